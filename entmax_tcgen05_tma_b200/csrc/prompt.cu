// prompt.cu -- causal attention over packed prompts with grouped heads: entmax_attn_prompt, and its softmax
// kernel.  (1.5-entmax and other alpha: the gather forward's PK instantiations, fwd.cu.)
//
// For row i of a sequence and its keys j <= i: S_ij = scale <Q_i, K_j>, P~ = 2^((S_ij - m_i) log2 e),
// l_i = sum P~, O_i = (sum P~ V_j) / l_i, tau_i = m_i + ln l_i, with m_i a reference that follows the row's
// running maximum.  Unlike the two-pass softmax forward (fwd_softmax.cu), which forms S twice and P in two
// bf16 parts, S is formed once: m rises with the blocks, and only where it would rise by more than
// 2^RAISE are O (in TMEM) and l brought to the new reference -- in practice in the first block or two -- so
// the correction costs next to nothing and P~ stays below 2^RAISE.
//
// A persistent CTA per SM takes pairs of 128-row tiles of one sequence and head, so that each K and V block
// loaded serves 256 rows.  Warps 0-3 and 4-7 are the softmax of the two tiles, a thread per row (no sum or
// maximum crosses threads); warp 8 loads by TMA through a ring that runs on across the pairs; warp 9 issues the
// products.  While one tile's scores are in its softmax, the tensor core works for the other tile: P~
// overwrites S in TMEM (S is in registers by then), O += P~ V, then S of the next block.
//
// What bounds it: one exponential a pair.  The special-function unit makes 16 a clock and SM, 128 x 128 pairs
// take 1024 clocks; S and P V take 128 and at most 256.  So EMULATED of every 32 are computed on the
// FMA units instead (f2exp2_poly).
//
// P~ enters P V as one bf16 number where O is bf16 (an error of at most 2^-8 a weight, the output's own
// rounding), and as three (24 bits, every exponential from the special-function unit) where O is fp32.
#include <cuda_bf16.h>
#include <math.h>
#include "../../include/entmax_cache.h"
#include "common.cuh"
#include "internal.h"

namespace entmax {
namespace {

constexpr int KB = 128;                      // keys of a block
constexpr int PAIR = 2 * TILE;               // rows of a work item
constexpr int NS = 4;                        // ring stages, a K and a V block each
constexpr int BLOCK16 = KB * HEAD_DIM * 2;   // 16 KiB
constexpr int W_LOAD = 8, W_MMA = 9, PROMPT_THREADS = 384;  // warps 10 and 11 only complete a warpgroup
// registers a thread: 168 at launch (384 threads), then 216 for the two softmax warpgroups, which hold a row's
// 128 scores, and 72 for the third: 216 + 216 + 72 = 3 * 168
constexpr int REGS_SOFTMAX = 216, REGS_OTHER = 72;
constexpr int GRID = 148;
constexpr int LIST = 1024;                   // work items of a CTA and launch
constexpr int MAX_SEQS = 4096, MAX_PAIRS = 4096;  // sequences of a call; pairs of a sequence (1 Mi tokens)
constexpr float RAISE = 8.f;                 // log2 units
constexpr int EMULATED = 8;                  // of every 32 exponentials
constexpr float LOG2E_F = 1.4426950408889634f, LN2_F = 0.6931471805599453f;

constexpr int O_Q = 0;                              // Q pairs, two buffers
constexpr int O_RING = O_Q + 2 * 2 * TILE_BYTES;    // NS x (K block, V block)
constexpr int O_LIST = O_RING + NS * 2 * BLOCK16;   // Item[LIST]
struct Item {
    int first, len, pair, head;
};
constexpr int O_CTL = O_LIST + LIST * (int)sizeof(Item);
struct Ctl {
    uint64_t q_full[2], q_empty[2];
    uint64_t k_full[NS], v_full[NS], kv_empty[NS];
    uint64_t s_full[2], p_ready[2], o_full[2], o_empty[2];
    uint32_t tmem_base;
    int abort_flag;
    int items;
    int n_q, n_kv;                 // loads issued, for the drain after an abort
    uint32_t last_bar, last_par;   // the MMA thread's last commit
};
constexpr int PROMPT_SMEM = O_CTL + (int)sizeof(Ctl) + 1024;
static_assert(PROMPT_SMEM <= 227 * 1024, "shared memory");
// while the work list is made, the ring holds the sequences' pair counts and the counts by size
static_assert((MAX_SEQS + 3 * (MAX_PAIRS + 2)) * 4 <= NS * 2 * BLOCK16, "list scratch");
// TMEM columns: S of tile w at 128 w, O at 256 + 64 w.  P~ lies over S: its bf16 pairs in columns 0 .. 63 of it, a
// second part in 64 .. 127; a third has columns of its own.
constexpr int TM_S = 0, TM_O = 256, TM_P3 = 384;

// Blocks of tile w of a pair: its last block holds the diagonal.
__device__ __forceinline__ int tile_blocks(const Item& it, int w) {
    const int tile = 2 * it.pair + w;
    return tile * TILE < it.len ? tile + 1 : 0;
}

// 2^x for two values x <= 127: x = n + f with n the nearest integer (adding and subtracting 1.5 * 2^23), 2^f on
// [-1/2, 1/2] by a polynomial of degree 4 fitted to the least relative error with 2^0 exact (iteratively
// reweighted least squares; 2.8e-6), and n added to its exponent.  x is taken as -127 where it is less, and
// 2^-127 comes out as 0: its exponent field is 0 and the polynomial is 1 there.
__device__ __forceinline__ uint64_t f2exp2_poly(uint64_t x) {
    float a, b;
    f2unpack(x, a, b);
    x = f2pack(fmaxf(a, -127.f), fmaxf(b, -127.f));
    const uint64_t magic = f2pack(12582912.f, 12582912.f);
    const uint64_t t = f2add(x, magic);
    const uint64_t f = f2sub(x, f2sub(t, magic));
    uint64_t p = f2pack(9.582852944731712e-3f, 9.582852944731712e-3f);
    p = f2fma(p, f, f2pack(5.5906426161527634e-2f, 5.5906426161527634e-2f));
    p = f2fma(p, f, f2pack(2.4024099111557007e-1f, 2.4024099111557007e-1f));
    p = f2fma(p, f, f2pack(6.931241750717163e-1f, 6.931241750717163e-1f));
    p = f2fma(p, f, f2pack(1.f, 1.f));
    float ta, tb;
    f2unpack(t, ta, tb);
    f2unpack(p, a, b);
    return f2pack(__uint_as_float(__float_as_uint(a) + (__float_as_uint(ta) << 23)),
                  __uint_as_float(__float_as_uint(b) + (__float_as_uint(tb) << 23)));
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Two fp32 values as three bf16 pairs: the top 16 bits, the top 16 bits of the rest, and its rest rounded.
__device__ __forceinline__ void f2split3(uint64_t v, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    float x, y;
    f2unpack(v, x, y);
    const uint32_t xt = __float_as_uint(x) & 0xffff0000u, yt = __float_as_uint(y) & 0xffff0000u;
    hi = __byte_perm(xt, yt, 0x7632);
    f2split(f2sub(v, f2pack(__uint_as_float(xt), __uint_as_float(yt))), mid, lo);
}

// The CTA's share of the work: all pairs of all sequences and heads, those with the most keys first (by
// pair number, then sequence, then head: the heads of a group run side by side and share K and V in L2),
// dealt in turns that change direction.  All threads; scratch: the ring.
__device__ __forceinline__ void make_list(const AttnArgs& a, long long first_item, Item* list, int* scratch, Ctl* ctl) {
    int* pairs = scratch;               // [n] pairs of the sequence, 0 where it is out of range
    int* more = scratch + MAX_SEQS;     // [P + 1] sequences with more than t pairs; first their counts
    int* before = more + MAX_PAIRS + 2; // [P + 1] pairs with a number above t
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int P = (a.max_len + PAIR - 1) / PAIR;
    for (int t = tid; t <= P; t += PROMPT_THREADS) more[t] = 0;
    __syncthreads();
    for (int i = tid; i < a.n_seqs; i += PROMPT_THREADS) {
        const int c0 = a.cu[i], c1 = a.cu[i + 1];
        const bool bad = c0 < 0 || c1 < c0 || c1 > a.T || c1 - c0 > a.max_len;
        if (bad && blockIdx.x == 0) atomicExch(a.arg_status, STATUS_BAD_ARG);
        const int p = bad ? 0 : (c1 - c0 + PAIR - 1) / PAIR;
        pairs[i] = p;
        atomicAdd(&more[p], 1);
    }
    __syncthreads();
    if (warp == 0) {  // more[t] = sum over p > t of the counts, before[t] = sum over u > t of more[u]
        int c1 = 0, c2 = 0;
        for (int base = P; base >= 0; base -= 32) {
            const int t = base - lane;  // lanes from high numbers to low
            const int h = t >= 0 ? more[t] : 0;
            int x = h;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            const int m = c1 + x - h;  // sequences with more than t pairs
            int z = m;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, z, o);
                if (lane >= o) z += y;
            }
            if (t >= 0) {
                more[t] = m;
                before[t] = c2 + z - m;
            }
            c1 += __shfl_sync(0xffffffffu, x, 31);
            c2 += __shfl_sync(0xffffffffu, z, 31);
        }
    }
    __syncthreads();
    const long long total = ((long long)before[0] + more[0]) * a.H;
    int n = 0;
    {
        const long long left = total - first_item;
        // turns q with an item for this CTA
        for (int q = 0; q < LIST; ++q) {
            const long long at = (long long)q * gridDim.x + ((q & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
            if (at >= left) {
                if ((long long)q * gridDim.x >= left) break;
                continue;  // only in the last turn
            }
            n = q + 1;
        }
    }
    for (int q = warp; q < n; q += PROMPT_THREADS / 32) {
        const long long at = first_item + (long long)q * gridDim.x + ((q & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        Item it{0, 0, 0, 0};
        if (at < total) {
            const int k = (int)(at / a.H);
            // the pair number: the highest t with before[t] + more[t] > k
            int lo = 0, hi = P;  // before[lo] + more[lo] > k
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (before[mid] + more[mid] > k) lo = mid;
                else hi = mid;
            }
            int rank = k - before[lo];  // among the sequences with more than lo pairs
            int s = -1;
            for (int i0 = 0; i0 < a.n_seqs && s < 0; i0 += 32) {
                const int i = i0 + lane;
                const uint32_t m = __ballot_sync(0xffffffffu, i < a.n_seqs && pairs[i] > lo);
                const int c = __popc(m);
                if (rank < c) s = i0 + __fns(m, 0, rank + 1);
                rank -= c;
            }
            it.first = a.cu[s];
            it.len = a.cu[s + 1] - it.first;
            it.pair = lo;
            it.head = (int)(at - (long long)k * a.H);
        }
        if (lane == 0) list[q] = it;
    }
    if (tid == 0) ctl->items = n;
}

template <bool kF32>
__global__ void __launch_bounds__(PROMPT_THREADS, 1)
prompt_softmax_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v, const AttnArgs a, const FwdOut out, long long first_item) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sQ = smem + O_Q;
    uint8_t* ring = smem + O_RING;
    const Item* list = reinterpret_cast<const Item*>(smem + O_LIST);
    Ctl* ctl = reinterpret_cast<Ctl*>(smem + O_CTL);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const WaitCfg wc{a.status, a.timeout_ns};

    if (tid == 0) {
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&ctl->q_full[b]), 1);
            mbar_init(smem_u32(&ctl->q_empty[b]), 1);
            mbar_init(smem_u32(&ctl->s_full[b]), 1);
            mbar_init(smem_u32(&ctl->p_ready[b]), 4);
            mbar_init(smem_u32(&ctl->o_full[b]), 1);
            mbar_init(smem_u32(&ctl->o_empty[b]), 4);
        }
        for (int s = 0; s < NS; ++s) {
            mbar_init(smem_u32(&ctl->k_full[s]), 1);
            mbar_init(smem_u32(&ctl->v_full[s]), 1);
            mbar_init(smem_u32(&ctl->kv_empty[s]), 1);
        }
        ctl->abort_flag = 0;
        ctl->n_q = ctl->n_kv = 0;
        ctl->last_bar = ctl->last_par = 0;
        fence_barrier_init();
        prefetch_tmap(&map_q);
        prefetch_tmap(&map_k);
        prefetch_tmap(&map_v);
    }
    if (warp == W_LOAD) {
        tmem_alloc(smem_u32(&ctl->tmem_base), 512);
        tmem_relinquish();
    }
    make_list(a, first_item, reinterpret_cast<Item*>(smem + O_LIST), reinterpret_cast<int*>(ring), ctl);
    fence_proxy_async_smem();  // the scratch gives way to TMA writes
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    const int items = ctl->items;

    if (warp >= W_LOAD) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
    if (warp == W_LOAD) {
        if (lane == 0) {
            int n_kv = 0, n_q = 0;
            bool ok = true;
            for (int q = 0; q < items && ok; ++q) {
                const Item it = list[q];
                const int nb0 = tile_blocks(it, 0), nb1 = tile_blocks(it, 1), nb = max(nb0, nb1);
                if (nb == 0) continue;
                const int kvh = it.head / (a.H / a.Hkv);
                const int qb = n_q & 1;
                ok = wait_bounded(smem_u32(&ctl->q_empty[qb]), ((uint32_t)(n_q >> 1) & 1u) ^ 1u, &ctl->abort_flag, wc);
                if (!ok) break;
                mbar_arrive_expect_tx(smem_u32(&ctl->q_full[qb]), (nb1 ? 2 : 1) * TILE_BYTES);
                const int row0 = it.first + it.pair * PAIR;
                tma_load_3d(smem_u32(sQ + qb * 2 * TILE_BYTES), &map_q, 0, it.head, row0, smem_u32(&ctl->q_full[qb]));
                if (nb1)
                    tma_load_3d(smem_u32(sQ + (qb * 2 + 1) * TILE_BYTES), &map_q, 0, it.head, row0 + TILE,
                                smem_u32(&ctl->q_full[qb]));
                ctl->n_q = ++n_q;
                for (int j = 0; j < nb; ++j) {
                    const int st = n_kv % NS;
                    ok = wait_bounded(smem_u32(&ctl->kv_empty[st]), ((uint32_t)(n_kv / NS) & 1u) ^ 1u, &ctl->abort_flag, wc);
                    if (!ok) break;
                    uint8_t* kb = ring + st * 2 * BLOCK16;
                    mbar_arrive_expect_tx(smem_u32(&ctl->k_full[st]), BLOCK16);
                    tma_load_3d(smem_u32(kb), &map_k, 0, kvh, it.first + j * KB, smem_u32(&ctl->k_full[st]));
                    mbar_arrive_expect_tx(smem_u32(&ctl->v_full[st]), BLOCK16);
                    tma_load_3d(smem_u32(kb + BLOCK16), &map_v, 0, kvh, it.first + j * KB, smem_u32(&ctl->v_full[st]));
                    ctl->n_kv = ++n_kv;
                }
            }
        }
        __syncwarp();
    } else if (warp == W_MMA) {
        if (lane == 0) {
            constexpr uint32_t IDESC_S = umma_idesc_bf16_f32(TILE, KB);
            constexpr uint32_t IDESC_O = umma_idesc_bf16_f32_bmn(TILE, HEAD_DIM);
            uint32_t last_bar = 0, last_par = 0;
            int n_kv = 0, n_q = 0;
            int ns[2] = {0, 0}, no[2] = {0, 0};  // score blocks and items of each tile so far
            bool ok = true;
            auto commit = [&](uint64_t* bar, uint32_t par) {
                tc_commit(smem_u32(bar));
                last_bar = smem_u32(bar);
                last_par = par;
            };
            for (int q = 0; q < items && ok; ++q) {
                const Item it = list[q];
                const int nbw[2] = {tile_blocks(it, 0), tile_blocks(it, 1)};
                const int nb = max(nbw[0], nbw[1]);
                if (nb == 0) continue;
                const int qb = n_q & 1;
                ok = wait_bounded(smem_u32(&ctl->q_full[qb]), (uint32_t)(n_q >> 1) & 1u, &ctl->abort_flag, wc);
                if (!ok) break;
                // step j: P V of block j - 1, then S of block j, for one tile after the other
                for (int j = 0; j <= nb && ok; ++j) {
                    const int st = (n_kv + j) % NS, pst = (n_kv + j + NS - 1) % NS;
                    if (j < nb) ok = wait_bounded(smem_u32(&ctl->k_full[st]), (uint32_t)((n_kv + j) / NS) & 1u, &ctl->abort_flag, wc);
                    if (ok && j > 0)
                        ok = wait_bounded(smem_u32(&ctl->v_full[pst]), (uint32_t)((n_kv + j - 1) / NS) & 1u, &ctl->abort_flag, wc);
                    if (!ok) break;
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const uint32_t s_tm = tmem + TM_S + 128u * w, o_tm = tmem + TM_O + 64u * w;
                        if (j > 0 && j <= nbw[w]) {
                            if (j == 1)  // O of the item before is read
                                ok = ok && wait_bounded(smem_u32(&ctl->o_empty[w]), ((uint32_t)no[w] & 1u) ^ 1u, &ctl->abort_flag, wc);
                            ok = ok && wait_bounded(smem_u32(&ctl->p_ready[w]), (uint32_t)(ns[w] - 1) & 1u, &ctl->abort_flag, wc);
                            if (!ok) break;
                            tc_fence_after();
                            const uint64_t vm = umma_desc_mnmajor_sw128(smem_u32(ring + pst * 2 * BLOCK16 + BLOCK16));
#pragma unroll
                            for (int k = 0; k < KB / 16; ++k)
                                tc_mma_bf16_ta(o_tm, s_tm + 8 * k, vm + 128u * k, IDESC_O, (j > 1 || k > 0) ? 1u : 0u);
                            if (kF32) {
#pragma unroll
                                for (int k = 0; k < KB / 16; ++k)
                                    tc_mma_bf16_ta(o_tm, s_tm + 64 + 8 * k, vm + 128u * k, IDESC_O, 1u);
#pragma unroll
                                for (int k = 0; k < KB / 16; ++k)
                                    tc_mma_bf16_ta(o_tm, tmem + TM_P3 + 64u * w + 8 * k, vm + 128u * k, IDESC_O, 1u);
                            }
                            if (j == nbw[w]) {
                                commit(&ctl->o_full[w], (uint32_t)no[w] & 1u);
                                ++no[w];
                            }
                        }
                        if (j < nbw[w]) {
                            tc_fence_after();
                            const uint64_t dq = umma_desc_kmajor_sw128(smem_u32(sQ + (qb * 2 + w) * TILE_BYTES));
                            const uint64_t dk = umma_desc_kmajor_sw128(smem_u32(ring + st * 2 * BLOCK16));
#pragma unroll
                            for (int k = 0; k < HEAD_DIM / 16; ++k) tc_mma_bf16(s_tm, dq + 2u * k, dk + 2u * k, IDESC_S, k > 0 ? 1u : 0u);
                            commit(&ctl->s_full[w], (uint32_t)ns[w] & 1u);
                            ++ns[w];
                        }
                    }
                    if (!ok) break;
                    if (j > 0) commit(&ctl->kv_empty[pst], (uint32_t)((n_kv + j - 1) / NS) & 1u);
                }
                if (!ok) break;
                commit(&ctl->q_empty[qb], (uint32_t)(n_q >> 1) & 1u);
                n_kv += nb;
                ++n_q;
            }
            ctl->last_bar = last_bar;
            ctl->last_par = last_par;
        }
        __syncwarp();
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
        // softmax of tile w: thread <-> row r of the tile <-> TMEM lane
        const int w = warp >> 2, r = tid & (TILE - 1);
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_tm = tmem + lanes + TM_S + 128u * w, o_tm = tmem + lanes + TM_O + 64u * w;
        const float c = a.scale * LOG2E_F, raise = RAISE / c;
        const uint64_t c2 = f2pack(c, c);
        int ns = 0, no = 0, n_kv = 0;
        bool live = true;
        for (int q = 0; q < items && live; ++q) {
            const Item it = list[q];
            const int nb = tile_blocks(it, w), nb_all = max(tile_blocks(it, 0), tile_blocks(it, 1));
            const int i = (2 * it.pair + w) * TILE + r;
            float m = -INFINITY;
            uint64_t l2 = 0, l3 = 0;
            for (int j = 0; j < nb; ++j) {
                live = __all_sync(0xffffffffu, wait_bounded(smem_u32(&ctl->s_full[w]), (uint32_t)ns & 1u, &ctl->abort_flag, wc));
                if (!live) break;
                ++ns;
                tc_fence_after();
                float v[4][32];
#pragma unroll
                for (int k = 0; k < 4; ++k) tmem_ld32(s_tm + 32 * k, v[k]);
#pragma unroll
                for (int k = 0; k < 4; ++k) tmem_wait_ld(v[k]);
                const bool diag = j == nb - 1;
                if (diag) {  // keys behind the row
                    const int lim = i - j * KB;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (32 * k + e > lim) v[k][e] = -INFINITY;
                }
                const float top = fmaxf(fmaxf(max32(v[0]), max32(v[1])), fmaxf(max32(v[2]), max32(v[3])));
                if (j == 0) {
                    m = top == -INFINITY ? 0.f : top;  // -inf: infinite inputs only (key 0 is every row's)
                } else if (__any_sync(0xffffffffu, top > m + raise)) {
                    // O and l to the new reference, row by row (a row's numbers do not depend on its neighbours).  S
                    // of this block was issued behind P V of the last, so O is at rest
                    const float n = top > m + raise ? top : m, f = ex2((m - n) * c);
                    m = n;
                    const uint64_t f2 = f2pack(f, f);
                    l2 = f2mul(l2, f2);
                    l3 = f2mul(l3, f2);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float o[32];
                        uint32_t u[32];
                        tmem_ld32(o_tm + 32 * k, o);
                        tmem_wait_ld(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(o[e] * f);
                        tmem_st32(o_tm + 32 * k, u);
                    }
                }
                const float off = -m * c;
                const uint64_t off2 = f2pack(off, off);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t hi[16], mid[16], lo[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const uint64_t x = f2fma(f2pack(v[k][e], v[k][e + 1]), c2, off2);
                        uint64_t p;
                        if (!kF32 && (e / 2) % (32 / EMULATED) == 0) {
                            p = f2exp2_poly(x);
                        } else {
                            float x0, x1;
                            f2unpack(x, x0, x1);
                            p = f2pack(ex2(x0), ex2(x1));
                        }
                        if (e & 2) l3 = f2add(l3, p);
                        else l2 = f2add(l2, p);
                        if (kF32) {
                            f2split3(p, hi[e >> 1], mid[e >> 1], lo[e >> 1]);
                        } else {
                            float x0, x1;
                            f2unpack(p, x0, x1);
                            hi[e >> 1] = pack_bf16(x0, x1);
                        }
                    }
                    tmem_st16(s_tm + 16 * k, hi);
                    if (kF32) {
                        tmem_st16(s_tm + 64 + 16 * k, mid);
                        tmem_st16(tmem + lanes + TM_P3 + 64u * w + 16 * k, lo);
                    }
                }
                tmem_wait_st();
                if (diag && j == nb_all - 1) {
                    // the rows of V behind the sequence's end belong to others: they must not reach P V, not even
                    // times 0 (they may be infinite or NaN).  This tile alone reads this block.
                    const int live_rows = it.len - j * KB;
                    if (live_rows < KB) {
                        const int st = (n_kv + j) % NS;
                        live = __all_sync(0xffffffffu, wait_bounded(smem_u32(&ctl->v_full[st]), (uint32_t)((n_kv + j) / NS) & 1u,
                                                                    &ctl->abort_flag, wc));
                        if (!live) break;
                        if (r >= live_rows) {
                            uint4* row = reinterpret_cast<uint4*>(ring + st * 2 * BLOCK16 + BLOCK16 + r * 128);
#pragma unroll
                            for (int k = 0; k < 8; ++k) row[k] = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl->p_ready[w]));
            }
            if (nb > 0 && live) {
                live = __all_sync(0xffffffffu, wait_bounded(smem_u32(&ctl->o_full[w]), (uint32_t)no & 1u, &ctl->abort_flag, wc));
                if (!live) break;
                ++no;
                tc_fence_after();
                float o[2][32];
                tmem_ld32(o_tm, o[0]);
                tmem_ld32(o_tm + 32, o[1]);
                tmem_wait_ld(o[0]);
                tmem_wait_ld(o[1]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl->o_empty[w]));
                float x0, x1, x2, x3;
                f2unpack(l2, x0, x1);
                f2unpack(l3, x2, x3);
                const float l = (x0 + x1) + (x2 + x3), inv = 1.f / l;
                if (i < it.len) {
                    const size_t t = (size_t)(it.first + i);
                    out.tau[(size_t)it.head * a.T + t] = (m * c + log2f(l)) * LN2_F;
                    const size_t at = (t * a.H + it.head) * HEAD_DIM;
                    if (kF32) {
                        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(out.O) + at);
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            dst[k] = make_float4(o[k >> 3][4 * (k & 7)] * inv, o[k >> 3][4 * (k & 7) + 1] * inv,
                                                 o[k >> 3][4 * (k & 7) + 2] * inv, o[k >> 3][4 * (k & 7) + 3] * inv);
                    } else {
                        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out.O) + at);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float* p = &o[k >> 2][8 * (k & 3)];
                            dst[k] = make_uint4(pack_bf16(p[0] * inv, p[1] * inv), pack_bf16(p[2] * inv, p[3] * inv),
                                                pack_bf16(p[4] * inv, p[5] * inv), pack_bf16(p[6] * inv, p[7] * inv));
                        }
                    }
                }
            }
            n_kv += nb_all;
        }
    }

    tc_fence_before();
    __syncthreads();
    // Past this barrier no thread waits, so the abort flag is final (uniform).  After an abort every TMA load
    // and MMA issued must complete before the CTA frees TMEM and its shared memory.
    if (flag_set(&ctl->abort_flag)) {
        if (lane == 0 && warp == W_LOAD) {
            for (int n = max(0, ctl->n_q - 2); n < ctl->n_q; ++n) wait_drain(smem_u32(&ctl->q_full[n & 1]), (uint32_t)(n >> 1) & 1u);
            for (int n = max(0, ctl->n_kv - NS); n < ctl->n_kv; ++n) {
                wait_drain(smem_u32(&ctl->k_full[n % NS]), (uint32_t)(n / NS) & 1u);
                wait_drain(smem_u32(&ctl->v_full[n % NS]), (uint32_t)(n / NS) & 1u);
            }
        }
        if (lane == 0 && warp == W_MMA && ctl->last_bar) wait_drain(ctl->last_bar, ctl->last_par);
        tc_fence_before();
        __syncthreads();
    }
    if (warp == W_LOAD) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace

cudaError_t launch_prompt_softmax(const AttnArgs& a, const FwdOut& o, cudaStream_t stream) {
    CUtensorMap mq, mk, mv;
    cudaError_t e = make_packed_map(&mq, a.Q, a.H, 64ll * a.q_step, a.T, TILE);
    if (e == cudaSuccess) e = make_packed_map(&mk, a.K, a.Hkv, 64ll * a.k_step, a.T, KB);
    if (e == cudaSuccess) e = make_packed_map(&mv, a.V, a.Hkv, 64ll * a.v_step, a.T, KB);
    if (e != cudaSuccess) return e;
    const auto f = o.out_f32 ? prompt_softmax_kernel<true> : prompt_softmax_kernel<false>;
    e = ensure_smem_attr(reinterpret_cast<const void*>(f), PROMPT_SMEM, o.out_f32 ? 21 : 22);
    if (e != cudaSuccess) return e;
    // at most this many pairs; a CTA lists LIST of them
    const long long most = unit_base(a.T, a.n_seqs, PAIR, PAIR - 1) * a.H;
    const int grid = (int)(most < GRID ? (most < 1 ? 1 : most) : GRID);
    for (long long first = 0; first < most || first == 0; first += (long long)grid * LIST) {
        f<<<grid, PROMPT_THREADS, PROMPT_SMEM, stream>>>(mq, mk, mv, a, o, first);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace entmax

using namespace entmax;

extern "C" int entmax_attn_prompt(const void* Q, long long q_stride, const void* K, long long k_stride, const void* V,
                                  long long v_stride, const int32_t* cu, int n, int T, int max_len, float scale,
                                  float alpha, int H, int H_kv, int D, void* O, int out_dtype, float* tau,
                                  cudaStream_t stream) {
    if (n < 0 || T < 0 || max_len < 0 || H < 0 || H_kv < 0) return ENTMAX_ERR_ARG;
    if (!(scale > 0.f) || !isfinite(scale)) return ENTMAX_ERR_ARG;
    const bool soft = fabsf(alpha - 1.f) < 1e-4f;
    if (!soft && !(alpha > 1.f && alpha <= 2.f)) return ENTMAX_ERR_ARG;
    if (D != HEAD_DIM) return ENTMAX_ERR_UNSUPPORTED;
    if (out_dtype != ENTMAX_BF16 && out_dtype != ENTMAX_F32) return ENTMAX_ERR_ARG;
    if (H == 0 || H_kv == 0) return H == H_kv ? ENTMAX_OK : ENTMAX_ERR_ARG;
    if (H % H_kv != 0) return ENTMAX_ERR_ARG;
    if (n > MAX_SEQS || H > 65535 || max_len > (soft ? MAX_PAIRS * PAIR : MAX_L)) return ENTMAX_ERR_UNSUPPORTED;
    if (n == 0 || T == 0 || max_len == 0) return ENTMAX_OK;
    if (!Q || !K || !V || !O || !tau || !cu) return ENTMAX_ERR_ARG;
    if (!aligned(Q, 16) || !aligned(K, 16) || !aligned(V, 16) || !aligned(O, 16) || !aligned(tau, 4) || !aligned(cu, 4))
        return ENTMAX_ERR_ARG;
    if (q_stride % 64 || k_stride % 64 || v_stride % 64 || q_stride < 64ll * H || k_stride < 64ll * H_kv ||
        v_stride < 64ll * H_kv)
        return ENTMAX_ERR_ARG;
    if (q_stride > (1ll << 36) || k_stride > (1ll << 36) || v_stride > (1ll << 36)) return ENTMAX_ERR_UNSUPPORTED;
    int *status = nullptr, *args_status = nullptr;
    int rc = abi_record(abi_status_ptr(&status));
    if (!rc) rc = abi_record(serving_status_ptr(&args_status));
    if (rc) return rc;
    AttnArgs a{Q, K, V, nullptr, 1, H, 0, 1, 0, scale, status, abi_timeout_ns(), H_kv, soft ? 0.f : alpha - 1.f, 1};
    a.cu = cu;
    a.n_seqs = n;
    a.T = T;
    a.max_len = max_len;
    a.q_step = (int)(q_stride / 64);
    a.k_step = (int)(k_stride / 64);
    a.v_step = (int)(v_stride / 64);
    a.arg_status = args_status;
    const FwdOut o{O, out_dtype == ENTMAX_F32, tau, SavedSupport{}, nullptr, nullptr};
    return abi_record(soft ? launch_prompt_softmax(a, o, stream) : launch_fwd_packed(a, o, stream));
}
