// moe_lora_matmul: a shared projection and each token's low-rank adapter in one product.
//
//   y[t] = W x_t + B_a u_t,   u_t = scale[a] A_a x_t,   a = adapter[t]
// Two kernels.  lora_shrink_kernel computes u in fp32 and leaves it as two 16-bit halves (the nearest, and the nearest of what
// is left: 16 bits of bf16, 22 of fp16), 32 ranks to a 128-byte row piece, upper halves first (and, where a third part is kept,
// another piece for it).  fp16 lacks the range for that.  The product of few rows takes u in fp32 instead, as two halves of tf32.  For
// the other one a token's ranks (T <= LS_FEW: each 32 of them) are first brought to the top of fp16's range by a power of two, whose
// reciprocal is kept behind u, and the product undoes it.  For 16-bit results only where the largest is below 1/8 (above, its
// elements are off by 2^-22 of it at most as they are): the adapter's part then wants an accumulator of its own, in which the next
// item can't begin (4096 tokens, rank 32: 52 us, 58 for small u).  The product's kernel (moe_grouped.cuh, GP_LORA) runs K on into
// the ranks: for each adapter that has tokens in its tile, 32 ranks at a time, B_a's tile against the tokens' rows of u, zeros for the
// tokens of other adapters.  So y is rounded once, and W's part and the adapters' share an accumulator or are added before that.
// The product starts beside the first kernel and waits for u only where it loads it.
#include <algorithm>
#include <mutex>

#include "moe_grouped.cuh"

namespace {

#define LS_RANKS 4         // few tokens: ranks of a warp
#define LS_FEW 64          // tokens

template <bool BF>
__device__ __forceinline__ float2 pair_value(uint32_t w) {
    if (BF) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*(const __half2 *)&w);
}
// fp16's powers of two: what of v is finite in fp16 counts, and the largest of it, where that is below `below`, comes to 2^14 or
// more (below 2^-86: to less).
__device__ __forceinline__ float finite16(float v) { return fabsf(v) < 65520.f ? fabsf(v) : 0.f; }
__device__ __forceinline__ void power16(float most, float below, float &up, float &down) {
    const int e = most > 0.f && most < below ? max((int)(__float_as_uint(most) >> 23) - 127 - 14, -100) : 0;
    up = __uint_as_float((uint32_t)(127 - e) << 23);
    down = __uint_as_float((uint32_t)(127 + e) << 23);
}
// v (fp16: times `up`) as two 16-bit numbers (one that overflows: as the infinity alone).
// (rest: what they leave, as a third.)
template <bool BF>
__device__ __forceinline__ void split16(float v, float up, uint16_t &hi, uint16_t &lo, uint16_t &rest) {
    if (BF) {
        const __nv_bfloat16 h = __float2bfloat16_rn(v);
        const float f = __bfloat162float(h), left = isinf(f) ? 0.f : v - f;
        const __nv_bfloat16 l = __float2bfloat16_rn(left);
        hi = __bfloat16_as_ushort(h);
        lo = __bfloat16_as_ushort(l);
        rest = __bfloat16_as_ushort(__float2bfloat16_rn(left - __bfloat162float(l)));
    } else {
        const bool in = fabsf(v) < 65520.f;
        const __half h = __float2half_rn(in ? v * up : v);
        hi = __half_as_ushort(h);
        lo = __half_as_ushort(__float2half_rn(in ? v * up - __half2float(h) : 0.f));
        rest = 0;
    }
}

// Few tokens: a warp for LS_RANKS ranks of one token, a CTA for 32 of them.  Next to no shared memory: it runs beside the product.
// u: [T][chunks][parts][64], fp16: and factor [T][chunks].  F32: u as it is, [T][chunks][32].
template <bool BF, bool F32>
__global__ void __launch_bounds__(256) lora_shrink_kernel(const uint16_t *x, size_t ldx, int T, int K, const int32_t *adapter,
                                                          int n_adapters, const uint16_t *a, int rank, const float *scale,
                                                          uint16_t *u, float *factor, float below, int parts) {
    __shared__ float most[8];  // (fp16)
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x % 32, chunks = (rank + 31) / 32, groups = chunks * 32 / LS_RANKS;
    const long long job = (long long)blockIdx.x * 8 + threadIdx.x / 32;
    const int t = (int)(job / groups), j0 = (int)(job % groups) * LS_RANKS;
    if (t >= T) return;
    const int ad = adapter[t];
    if (ad < 0 || ad >= n_adapters) return;  // (no product reads this row)
    float v[LS_RANKS] = {};
    if (j0 < rank) {
        const uint16_t *xr = x + (size_t)t * ldx, *ar = a + ((size_t)ad * rank + j0) * K;
        for (int k0 = 0; k0 < K; k0 += 2048) {  // (sums of 64 products a lane, and their sum: K = 65536 in one go 8e-7 off)
            float part[LS_RANKS] = {};
            const int end = min(K, k0 + 2048);
#pragma unroll 4
            for (int k = k0 + 8 * lane; k < end; k += 256) {  // (several turns' loads in flight)
                const uint4 xv = __ldg((const uint4 *)(xr + k));
                const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
                uint4 avs[LS_RANKS];
#pragma unroll
                for (int j = 0; j < LS_RANKS; ++j) avs[j] = __ldg((const uint4 *)(ar + (size_t)j * K + k));
#pragma unroll
                for (int j = 0; j < LS_RANKS; ++j) {  // (the rank is a multiple of 8)
                    const uint4 av = avs[j];
                    const uint32_t aw[4] = {av.x, av.y, av.z, av.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 p = pair_value<BF>(xw[i]), q = pair_value<BF>(aw[i]);
                        part[j] = fmaf(p.x, q.x, part[j]);
                        part[j] = fmaf(p.y, q.y, part[j]);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < LS_RANKS; ++j) v[j] += part[j];
        }
#pragma unroll
        for (int j = 0; j < LS_RANKS; ++j)
#pragma unroll
            for (int d = 16; d > 0; d /= 2) v[j] += __shfl_xor_sync(0xffffffffu, v[j], d);
    }
    float up = 1.f, down = 1.f;
    if (!BF && !F32) {  // (a CTA's warps have the same token)
        float m = 0.f;
        const float sc = scale ? scale[ad] : 1.f;
#pragma unroll
        for (int j = 0; j < LS_RANKS; ++j) m = fmaxf(m, finite16(v[j] * sc));
        if (lane == 0) most[threadIdx.x / 32] = m;
        __syncthreads();
        for (int w = 0; w < 8; ++w) m = fmaxf(m, most[w]);
        power16(m, below, up, down);
        // (32 ranks of zeros: the smallest, which is none of the token's other ranks' largest)
        if (threadIdx.x == 0) factor[(size_t)t * chunks + j0 / 32] = m > 0.f ? down : 0x1p-100f;
    }
    if (lane < LS_RANKS) {
        float r = 0.f;
#pragma unroll
        for (int j = 0; j < LS_RANKS; ++j)
            if (j == lane) r = v[j];
        if (scale) r *= scale[ad];
        if (j0 >= rank) r = 0.f;
        uint16_t hi, lo, rest;
        split16<BF>(r, up, hi, lo, rest);
        const int j = j0 + lane;
        if (F32) {
            ((float *)u)[(size_t)t * chunks * 32 + j] = fabsf(r) < 65520.f ? r : __half2float(__float2half_rn(r));
            return;
        }
        uint16_t *row = u + ((size_t)t * chunks + j / 32) * parts * 64 + j % 32;
        row[0] = hi;
        row[32] = lo;
        if (parts == 2) {
            row[64] = rest;
            row[96] = 0;
        }
    }
}

#define LS_TOKENS 128      // tokens of a tile: the M side of the MMA
#define LS_COLS 256        // most ranks of a pass, of one adapter or several: its N side
#define LS_STAGES 4
#define LS_STAGE (LS_TOKENS * 128 + LS_COLS * 128)  // 64 columns of x and of A
#define LS_THREADS 256
#define LS_HEADER 3072
#define LS_MAX_SPLIT 8     // CTAs (a cluster) that share a tile's K
#define LS_SMEM (1024 + LS_HEADER + LS_STAGES * LS_STAGE)

struct ShrinkParams {
    CUtensorMap x, a;  // x by boxes of 128 rows, A by adapters
    int T, K, rank, n_adapters, per_pass, fmt, parts;  // per_pass: adapters of a pass
    int acc_stages;    // most stages of an accumulator
    const int32_t *adapter;
    const float *scale;
    uint16_t *u;       // [T][chunks][parts][64]
    float *factor;     // [T][chunks], fp16
    float below;       // tokens whose largest is below this come by a power of two (fp16)
    int *status;
};

struct ShrinkSmem {
    uint64_t full[LS_STAGES], empty[LS_STAGES], acc_full[2], acc_empty[2], done;
    uint32_t tmem;
    int abort;
    int count[LS_TOKENS / 32];
    alignas(16) int ids[LS_TOKENS];  // adapter of each token, -1: none
    int place[LS_TOKENS];            // of a token that is its adapter's first: the adapter's place among the tile's
    int list[LS_TOKENS];             // adapter of each place
    unsigned most[LS_TOKENS];        // fp16: bits of the largest of each token's u
    int mine[LS_TOKENS];             // place of each token's adapter in this pass, -1: not in it
};
static_assert(sizeof(ShrinkSmem) <= LS_HEADER, "");

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// Many tokens.  A cluster: a tile of 128 tokens, one pass over some of its adapters (blockIdx.y); its CTAs share K.
// D[token][rank] on the tensor cores, x the M side, the rows of the pass's A_a one after another the N side; a token keeps
// its own adapter's columns.  The CTAs' sums are added up in the order of their ranks, each CTA for its share of the tokens.
template <bool BF>
__global__ void __launch_bounds__(LS_THREADS, 1) lora_shrink_mma_kernel(const __grid_constant__ ShrinkParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_smem_1024(smem_raw), *ring = smem + LS_HEADER;
    ShrinkSmem &s = *(ShrinkSmem *)smem;
    static_assert(LS_TOKENS * (MOE_MAX_RANK + 4) * 4 <= LS_STAGES * LS_STAGE, "sums in the ring's place");
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int ctas = (int)cluster_nctarank(), me = (int)cluster_ctarank();
    const int t0 = (int)blockIdx.x / ctas * LS_TOKENS, n = min(LS_TOKENS, p.T - t0), chunks = (p.rank + 31) / 32;
    if (tid == 0) {
        for (int i = 0; i < LS_STAGES; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.acc_full[i], 1);
            mbar_init(&s.acc_empty[i], LS_TOKENS / 32);
        }
        mbar_init(&s.done, 1);
        s.abort = 0;
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc_group<1>(&s.tmem, 2 * LS_COLS);  // two accumulators: see moe_grouped.cuh
    pdl_wait();
    pdl_trigger();
    // ---------------- the tile's adapters, in the order of their first tokens
    if (tid < LS_TOKENS) {
        const int a = tid < n ? p.adapter[t0 + tid] : -1;
        s.ids[tid] = a >= 0 && a < p.n_adapters ? a : -1;  // (others: recorded by the product)
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int head = -1;  // the first token of this token's adapter
    if (tid < LS_TOKENS) {
        const int a = s.ids[tid];
        if (a >= 0)
#pragma unroll 8
            for (int i = LS_TOKENS - 4; i >= 0; i -= 4) {
                const int4 v = *(const int4 *)&s.ids[i];
                head = v.w == a ? i + 3 : head;
                head = v.z == a ? i + 2 : head;
                head = v.y == a ? i + 1 : head;
                head = v.x == a ? i : head;
            }
        const unsigned heads = __ballot_sync(0xffffffffu, head == tid);
        if (head == tid) s.place[tid] = __popc(heads & ((1u << lane) - 1u));
        if (lane == 0) s.count[warp] = __popc(heads);
    }
    __syncthreads();
    int all = 0, base = 0;
    for (int w = 0; w < LS_TOKENS / 32; ++w) {
        base += w < warp ? s.count[w] : 0;
        all += s.count[w];
    }
    if (tid < LS_TOKENS && head == tid) {
        s.place[tid] += base;
        s.list[s.place[tid]] = s.ids[tid];
    }
    __syncthreads();
    const int first = (int)blockIdx.y * p.per_pass, used = min(p.per_pass, all - first);
    const bool work = used > 0;  // (the same for the whole cluster)
    if (work) {
        int mine = -1;
        if (tid < LS_TOKENS) {
            if (head >= 0) mine = s.place[head] - first;
            if (mine >= used) mine = -1;
            s.mine[tid] = max(mine, -1);
        }
        const int KB = (p.K + 63) / 64, kb0 = KB * me / ctas, kb1 = KB * (me + 1) / ctas;
        // accumulators of `per` stages, in turn the first and the second half of tensor memory; of more than two, warps 0 to 3 add
        // each to the next one, and hand it back, while that one is filled (see moe_grouped.cuh)
        const int per = max(1, min(p.acc_stages, (kb1 - kb0 + 1) / 2)), accs = (kb1 - kb0 + per - 1) / per;
        if (warp == 4) {
            // ---------------- copies
            int st = 0;
            uint32_t ph = 1;
            bool ok = true;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (kb - kb0 >= LS_STAGES && !(ok = mbar_wait_warp(&s.empty[st], ph, p.status, &s.abort))) break;
                uint8_t *dst = ring + (size_t)st * LS_STAGE;
                const uint32_t bar = smem_u32(&s.full[st]);
                mbar_arrive_expect_tx_elect(&s.full[st], (uint32_t)(LS_TOKENS + used * p.rank) * 128u);
                if (lane == 0) tma_tile_2d<1>(dst, &p.x, kb * 64, t0, bar);
                if (lane < used)  // (at most 256 / 8)
                    tma_tile_3d<1>(dst + (LS_TOKENS + lane * p.rank) * 128, &p.a, kb * 64, 0, s.list[first + lane], bar);
                __syncwarp();
                if (++st == LS_STAGES) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            if (!ok) settle_after_abort();
        } else if (warp == 5) {
            // ---------------- MMAs
            int st = 0;
            uint32_t ph = 0;
            const uint32_t d0 = __shfl_sync(0xffffffffu, s.tmem, 0);
            const uint32_t idesc = umma_idesc_16(p.fmt, false, false, 128, __shfl_sync(0xffffffffu, (used * p.rank + 15) & ~15, 0));
            bool ok = true;
            for (int acc = 0, kb = kb0; acc < accs && ok; ++acc) {
                const uint32_t d = d0 + (acc & 1) * LS_COLS;
                if (acc >= 2 && !(ok = mbar_wait_warp(&s.acc_empty[acc & 1], (acc / 2 - 1) & 1, p.status, &s.abort))) break;
                const int from = kb;
                for (const int end = min(kb1, kb + per); kb < end; ++kb) {
                    if (!(ok = mbar_wait_warp(&s.full[st], ph, p.status, &s.abort))) break;
                    tc_fence_after();
                    const uint32_t sa = smem_u32(ring) + (uint32_t)st * LS_STAGE;
                    const uint64_t a = umma_desc_sw128(sa), b = umma_desc_sw128(sa + LS_TOKENS * 128);
                    const int left = p.K - 64 * kb;
                    umma_f16_elect<1>(d, a, b, idesc, kb > from);
                    if (left > 16) umma_f16_elect<1>(d, a + 2, b + 2, idesc, 1);
                    if (left > 32) umma_f16_elect<1>(d, a + 4, b + 4, idesc, 1);
                    if (left > 48) umma_f16_elect<1>(d, a + 6, b + 6, idesc, 1);
                    umma_commit_elect(&s.empty[st]);
                    if (++st == LS_STAGES) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
                if (ok && accs > 2) umma_commit_elect(&s.acc_full[acc & 1]);
            }
            umma_commit_elect(&s.done);  // every copy has been consumed, every MMA has completed
        } else if (warp < 4) {
            const uint32_t tb = s.tmem + ((uint32_t)(32 * warp) << 16);
            for (int acc = 0; acc + 2 < accs; ++acc) {
                if (!mbar_wait_warp(&s.acc_full[acc & 1], (acc / 2) & 1, p.status, &s.abort)) break;
                if (!mbar_wait_warp(&s.acc_full[(acc + 1) & 1], ((acc + 1) / 2) & 1, p.status, &s.abort)) break;
                tc_fence_after();
                const uint32_t from = tb + (acc & 1) * LS_COLS, to = tb + ((acc + 1) & 1) * LS_COLS;
                for (int i = 0; i < used; ++i) {
                    if (!__any_sync(0xffffffffu, mine == i)) continue;
                    for (int c = i * p.rank; c < (i + 1) * p.rank; c += 8) {
                        uint32_t v[8], w[8];
                        tmem_ld8(from + c, v);
                        tmem_ld8(to + c, w);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(__uint_as_float(v[k]) + __uint_as_float(w[k]));
                        tmem_st8(to + c, w);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive1(&s.acc_empty[acc & 1]);
            }
        }
        __syncwarp();
        const bool ok = mbar_wait_role(&s.done, 0, p.status, &s.abort);
        const bool fine = __syncthreads_and(ok);
        tc_fence_after();
        // ---------------- this CTA's sums: a token's own adapter's columns
        float *part = (float *)ring;  // [LS_TOKENS][rank + 4]
        const int pitch = p.rank + 4;
        if (fine && warp < 4) {
            const uint32_t tb = s.tmem + ((uint32_t)(32 * warp) << 16);
            float *o = part + (size_t)tid * pitch;
            for (int i = 0; i < used; ++i) {
                if (!__any_sync(0xffffffffu, mine == i)) continue;
                for (int c = 0; c < p.rank; c += 8) {
                    uint32_t v[8];
                    tmem_ld8(tb + i * p.rank + c, v);
                    tmem_ld_wait();
                    if (accs > 1) {
                        uint32_t w[8];
                        tmem_ld8(tb + LS_COLS + i * p.rank + c, w);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) + __uint_as_float(w[k]));
                    }
                    if (mine == i) {
                        if (kb0 == kb1)
#pragma unroll
                            for (int k = 0; k < 8; ++k) v[k] = 0u;
                        *(float4 *)(o + c) = make_float4(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]),
                                                         __uint_as_float(v[3]));
                        *(float4 *)(o + c + 4) = make_float4(__uint_as_float(v[4]), __uint_as_float(v[5]), __uint_as_float(v[6]),
                                                             __uint_as_float(v[7]));
                    }
                }
            }
        }
        tc_fence_before();
        cluster_sync_all();
        // ---------------- the cluster's
        const int ta = LS_TOKENS * me / ctas, tb = LS_TOKENS * (me + 1) / ctas, quads = chunks * 8;
        auto total = [&](int t, int j) -> float4 {  // of ranks j .. j + 3, in the order of the CTAs
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int c = 0; c < ctas; ++c) {
                const float4 w = ld_cluster_f32x4(cluster_map(part + (size_t)t * pitch + j, c));
                v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
            }
            const float sc = p.scale ? p.scale[s.ids[t]] : 1.f;
            return make_float4(v.x * sc, v.y * sc, v.z * sc, v.w * sc);
        };
        if (!BF) {  // the largest of each token first; the sums stay in this CTA's own place for its tokens, which no other CTA reads
            for (int t = tid; t < LS_TOKENS; t += LS_THREADS) s.most[t] = 0u;
            __syncthreads();
            for (int i = tid; i < (tb - ta) * quads; i += LS_THREADS) {
                const int t = ta + i / quads, j = 4 * (i % quads);
                if (s.mine[t] < 0 || j >= p.rank) continue;
                const float4 v = total(t, j);
                *(float4 *)(part + (size_t)t * pitch + j) = v;
                const float m = fmaxf(fmaxf(finite16(v.x), finite16(v.y)), fmaxf(finite16(v.z), finite16(v.w)));
                atomicMax(&s.most[t], __float_as_uint(m));  // (no negative numbers: ordered as their bits are)
            }
            __syncthreads();
        }
        for (int i = tid; i < (tb - ta) * quads; i += LS_THREADS) {
            const int t = ta + i / quads, j = 4 * (i % quads);
            if (s.mine[t] < 0) continue;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (j < p.rank) v = BF ? total(t, j) : *(const float4 *)(part + (size_t)t * pitch + j);
            float up = 1.f, down = 1.f;
            if (!BF) {
                power16(__uint_as_float(s.most[t]), p.below, up, down);
                if (j % 32 == 0) p.factor[(size_t)(t0 + t) * chunks + j / 32] = down;
            }
            uint16_t hi[4], lo[4], rest[4];
            split16<BF>(v.x, up, hi[0], lo[0], rest[0]);
            split16<BF>(v.y, up, hi[1], lo[1], rest[1]);
            split16<BF>(v.z, up, hi[2], lo[2], rest[2]);
            split16<BF>(v.w, up, hi[3], lo[3], rest[3]);
            uint16_t *row = p.u + ((size_t)(t0 + t) * chunks + j / 32) * p.parts * 64 + j % 32;
            if (p.parts == 2) {
                *(uint2 *)(row + 64) = make_uint2(rest[0] | (uint32_t)rest[1] << 16, rest[2] | (uint32_t)rest[3] << 16);
                *(uint2 *)(row + 96) = make_uint2(0, 0);
            }
            *(uint2 *)row = make_uint2(hi[0] | (uint32_t)hi[1] << 16, hi[2] | (uint32_t)hi[3] << 16);
            *(uint2 *)(row + 32) = make_uint2(lo[0] | (uint32_t)lo[1] << 16, lo[2] | (uint32_t)lo[3] << 16);
        }
        cluster_sync_all();  // (no CTA leaves while its sums are read)
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_group<1>(s.tmem, 2 * LS_COLS);
    }
}

int check(int T, int rank) {
    MOE_CHECK(T >= 0 && T <= 1 << 24 && rank >= 1);
    if (rank % 8 || rank > MOE_MAX_RANK) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

int shrink_few(const void *x, size_t ldx, int T, int K, int type, const int32_t *adapter, int n_adapters, const void *a,
               int rank, const float *scale, void *u, float *factor, float below, int parts, moe_stream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    const long long jobs = (long long)T * ((rank + 31) / 32 * 32 / LS_RANKS);
    moe_pdl_config(&cfg, attr, dim3((unsigned)((jobs + 7) / 8)), dim3(256), 0, moe_cuda_stream(s));
    MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, type == MOE_BF16 ? lora_shrink_kernel<true, false> : factor ? lora_shrink_kernel<false, false> : lora_shrink_kernel<false, true>,
                                    (const uint16_t *)x, ldx, T, K, adapter, n_adapters, (const uint16_t *)a, rank, scale,
                                    (uint16_t *)u, factor, below, parts));
    return MOE_OK;
}

int shrink_many(const void *x, size_t ldx, int T, int K, int type, const int32_t *adapter, int n_adapters, const void *a,
                int rank, const float *scale, void *u, float *factor, float below, int parts, int acc_stages,
                int *status, moe_stream_t s) {
    static std::mutex mu;
    static bool ready[64] = {false};
    int dev = -1, rc;
    const int n = grouped_sms();
    MOE_TRY_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= 64) return MOE_ERR_UNSUPPORTED;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[dev]) {
            MOE_TRY_CUDA(cudaFuncSetAttribute(lora_shrink_mma_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, LS_SMEM));
            MOE_TRY_CUDA(cudaFuncSetAttribute(lora_shrink_mma_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, LS_SMEM));
            ready[dev] = true;
        }
    }
    ShrinkParams p = {};
    {
        const uint64_t dims[2] = {(uint64_t)K, (uint64_t)T}, strides[1] = {(uint64_t)ldx * 2};
        const uint32_t box[2] = {64, LS_TOKENS};
        if ((rc = grouped_map(&p.x, type, 2, x, dims, strides, box, 128)) != MOE_OK) return rc;
    }
    {
        const uint64_t dims[3] = {(uint64_t)K, (uint64_t)rank, (uint64_t)n_adapters};
        const uint64_t strides[2] = {(uint64_t)K * 2, (uint64_t)K * rank * 2};
        const uint32_t box[3] = {64, (uint32_t)rank, 1};
        if ((rc = grouped_map(&p.a, type, 3, a, dims, strides, box, 128)) != MOE_OK) return rc;
    }
    p.T = T;
    p.K = K;
    p.rank = rank;
    p.n_adapters = n_adapters;
    p.per_pass = LS_COLS / rank;
    p.fmt = type == MOE_BF16;
    p.adapter = adapter;
    p.scale = scale;
    p.u = (uint16_t *)u;
    p.factor = factor;
    p.below = below;
    p.parts = parts;
    p.acc_stages = acc_stages;
    p.status = status;
    const int tiles = (T + LS_TOKENS - 1) / LS_TOKENS, most = std::min(n_adapters, LS_TOKENS);
    const int passes = (most + p.per_pass - 1) / p.per_pass;
    int ctas = 1;
    while (ctas < LS_MAX_SPLIT && tiles * ctas * 2 <= n && ctas * 2 * 64 <= K) ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    moe_pdl_config(&cfg, attr, dim3((unsigned)(tiles * ctas), (unsigned)passes), dim3(LS_THREADS), LS_SMEM, moe_cuda_stream(s));
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, type == MOE_BF16 ? lora_shrink_mma_kernel<true> : lora_shrink_mma_kernel<false>, p));
    return MOE_OK;
}

}  // namespace

extern "C" int moe_lora_workspace(int T, int rank, size_t *bytes) {
    MOE_CHECK(bytes);
    const int rc = check(T, rank);
    if (rc != MOE_OK) return rc;
    *bytes = (size_t)T * ((rank + 31) / 32) * 256;
    return MOE_OK;
}

extern "C" int moe_lora_matmul(const void *x, int type, int T, size_t ldx, const void *w, int N, int K,
                               const int32_t *adapter, int n_adapters, const void *a, const void *b, int rank,
                               const float *scale, void *y, int ytype, size_t ldy, void *workspace, size_t ws_bytes,
                               moe_stream_t s) {
    size_t need = 0;
    int rc = moe_lora_workspace(T, rank, &need);
    if (rc != MOE_OK) return rc;
    MOE_CHECK((type == MOE_BF16 || type == MOE_F16) && (ytype == MOE_F32 || ytype == MOE_BF16 || ytype == MOE_F16));
    MOE_CHECK(N >= 1 && K >= 1 && n_adapters >= 1);
    if (N % 8 || K % 8 || N > 1 << 16 || K > 1 << 16) return MOE_ERR_UNSUPPORTED;
    MOE_CHECK(ldx >= (size_t)K && ldx % 8 == 0 && ldx <= (size_t)1 << 32 && ldy >= (size_t)N && ldy % 8 == 0);
    if (T == 0) return MOE_OK;
    MOE_CHECK(x && w && adapter && a && b && y && workspace && ws_bytes >= need);
    MOE_CHECK((((uintptr_t)x | (uintptr_t)w | (uintptr_t)a | (uintptr_t)b | (uintptr_t)y) & 15) == 0);
    MOE_CHECK(((uintptr_t)workspace & 255) == 0);

    int *status = moe_status_word_device_ptr();
    // bf16 with fp32 results: u in three parts, 24 bits (two leave y 1.8e-6 off, relative to its norm, three 3e-7)
    const int parts = type == MOE_BF16 && ytype == MOE_F32 ? 2 : 1;
    const int acc_stages = ytype == MOE_F32 ? 4 : 64;
    const int chunks = (rank + 31) / 32;
    float *factor = (float *)((uint8_t *)workspace + (size_t)T * chunks * 128);  // (fp16: one part, half of the workspace)
    // few tokens, and no more rows of W than CTAs run at once (N = 2816: 1 token 12.1 -> 8.4 us, 32 tokens 20.2 -> 12.4 by the
    // kernel for few rows; N = 11264: 15.1 -> 14.9 and 21.1 -> 29.9)
    const bool few = T <= GF_MAX_R && (N + 15) / 16 <= 2 * grouped_sms();
    const float below = ytype == MOE_F32 ? 65536.f : 0.125f;
    rc = T <= LS_FEW ? shrink_few(x, ldx, T, K, type, adapter, n_adapters, a, rank, scale, workspace, few ? nullptr : factor, below, parts, s)
                     : shrink_many(x, ldx, T, K, type, adapter, n_adapters, a, rank, scale, workspace, factor, below, parts, acc_stages, status, s);
    if (rc != MOE_OK) return rc;
    if (few) {
        GroupedFewParams f = {};
        f.x = (const uint16_t *)x;
        f.w = (const uint16_t *)w;
        f.ldx = ldx;
        f.G = 1;
        f.R = T;
        f.x_share = 1;
        f.x_rows = T;
        f.y_rows = T;
        f.y = y;
        f.ldy = ldy;
        f.ytype = ytype;
        f.M = N;
        f.K = K;
        f.adapter = adapter;
        f.b = (const uint16_t *)b;
        f.u = (const uint16_t *)workspace;
        f.n_adapters = n_adapters;
        f.rank = rank;
        f.parts = parts;
        f.status = status;
        return grouped_few_launch(f, GP_LORA, type == MOE_BF16, moe_cuda_stream(s));
    }
    GroupedParams p = {};
    {
        const uint64_t dims[3] = {(uint64_t)K, (uint64_t)N, 1}, strides[2] = {(uint64_t)K * 2, (uint64_t)N * K * 2};
        const uint32_t box[3] = {64, 128, 1};
        if ((rc = grouped_map(&p.a, type, 3, w, dims, strides, box, 128)) != MOE_OK) return rc;
    }
    {
        const uint64_t dims[2] = {(uint64_t)K, (uint64_t)T}, strides[1] = {(uint64_t)ldx * 2};
        const uint32_t box[2] = {64, 16}, box64[2] = {64, 64};
        if ((rc = grouped_map(&p.b, type, 2, x, dims, strides, box, 128)) != MOE_OK) return rc;
        if ((rc = grouped_map(&p.b64, type, 2, x, dims, strides, box64, 128)) != MOE_OK) return rc;
    }
    {
        const uint64_t dims[3] = {(uint64_t)rank, (uint64_t)N, (uint64_t)n_adapters};
        const uint64_t strides[2] = {(uint64_t)rank * 2, (uint64_t)N * rank * 2};
        const uint32_t box[3] = {32, 128, 1};
        if ((rc = grouped_map(&p.ab, type, 3, b, dims, strides, box, 64)) != MOE_OK) return rc;
    }
    p.rows = (const uint16_t *)workspace;
    p.ld = (size_t)chunks * parts * 64;
    p.parts = parts;
    p.lora_b = (const uint16_t *)b;
    p.factor = factor;
    p.factors = T <= LS_FEW ? chunks : 1;
    p.G = 1;
    p.R = T;
    p.x_rows = T;
    p.y_rows = T;
    p.x_share = 1;
    p.y = y;
    p.ldy = ldy;
    p.M = N;
    p.K = K;
    p.adapter = adapter;
    p.n_adapters = n_adapters;
    p.rank = rank;
    p.fmt = type == MOE_BF16;
    p.status = status;

    // narrow tiles while they are one round of CTAs (64 tokens, N = 2816: 17.7 us against 25.4; 200 tokens 33.6 against 28.8)
    const bool wide = (T + 31) / 32 * ((N + 127) / 128) > grouped_sms();
    const int nt = !wide ? 32 : ytype == MOE_F32 ? 128 : 256;
    const long long tiles = (T + nt - 1) / nt;
    return grouped_launch(p, ytype, type == MOE_BF16 ? GP_LORA : GP_LORA_F16, wide, tiles * ((N + 127) / 128), (K + 63) / 64 + std::min(T, n_adapters) * chunks * parts,
                          moe_cuda_stream(s));
}
