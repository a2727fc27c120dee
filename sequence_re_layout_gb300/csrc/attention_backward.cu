// attention_backward.cu -- the gradients of attention with a window and sinks, on the
// tensor cores.
//
// Two kernels, each with its sum in tensor memory from the first tile to the last, so
// that nothing is added by atomics and results repeat:
//   dk, dv   128 keys a CTA, over the tiles of queries that see them, of every query
//            head that shares the key head.  Scores are taken transposed, keys along
//            tensor memory's lanes, so that P^T and dS^T lie there as the products dv +=
//            P^T dO and dk += dS^T Q want them:
//                S^T = K Q^T,   P^T = 2^(c S^T - lse),   dP^T = V dO^T,
//                dS^T = P^T (dP^T - D)
//   dq       128 queries at a time, over the tiles of keys that they see:
//                S = Q K^T,   dP = dO V^T,   dq += dS K
// A window leaves few tiles of keys to one of queries, so the dq kernel's CTAs, one an SM,
// walk tiles of queries: the next one's loads and first scores run under this one's end (2 x
// 8192 x 32 heads of 64, window 1024: 271 us; 309 with a CTA for each).
//
// That is seven products of a pair of tiles where one kernel with atomics needs five.
//
// In both, four warpgroups share a tile's columns, 32 each, a row a thread.  What bounds
// them is the chain of waits, loads, exponentials and stores of a pair of tiles, so the
// products of the next pair are issued as early as tensor memory allows:
//   - the dq kernel's S and dP are free as soon as they have been read (dS has two places of
//     its own);
//   - so are S^T and dP^T for heads of 64, where P^T and dS^T have places of their own (2 x
//     128 + 2 x 64 columns beside dk and dv);
//   - for heads of 128, P^T and dS^T take the places of S^T and dP^T.
//
// In the dkv kernel lse and D vary along a row.  They are taken off inside the products,
// by 16 more of K: each query's row has -lse / c and -D there, in four 16-bit parts each,
// and the keys' side has ones (for fp16, whose range is small, other powers of two) where
// they belong.
// As loads from shared memory, a value each, they took 1200 of 3000 cycles a pair of tiles.
//
// Where key tiles differ much in work (the sinks' keys are seen by every query, a causal
// mask's first ones by most), or there are few, several CTAs share the longest ones: their
// sums go to memory and another kernel adds them in order.
//
// fp16 has units of its own for P and dS (attention_common.cuh), which are taken off the sums at
// the end.  The units, and the largest |v|, which says with the largest |dO| whether dS can have been
// past the range, are made by two warps that do nothing else: 2 x 8192 x 32 heads of 64, window 1024,
// take 613 us in fp16 and 595 in bf16, or in fp16 without the units.
//
// As in the forward, a row that comes out infinite or NaN is computed again from the
// definition, where that can differ.
//
// Both kernels of 2 x 8192 x 32 heads of 64 over 8 take 570 us with a window of 1024 and 4
// sinks, 1680 us without a window (1.16 PFLOP/s of whole tiles' seven products): half of the
// issue slots and of the tensor cores' cycles, so what bounds them is still the chain of a pair
// of tiles.  2 x 16384 x 16 heads of 128, window 4096: 2430 us, 1.47 PFLOP/s; 73 % (dk, dv) and
// 58 % (dq, before the order of its products changed) of the tensor cores' cycles.
#include <cuda.h>

#include <algorithm>

#include "attention.cuh"
#include "attention_common.cuh"

namespace basp_fp8 {
namespace {

constexpr int kWays = 4, kCols = kTile / kWays;               // warpgroups of values, columns of each
constexpr int kValueWarps = 4 * kWays, kLoadWarp = kValueWarps, kIssueWarp = kLoadWarp + 1, kTmemWarp = kLoadWarp + 2;
constexpr int kBackThreads = 32 * kValueWarps + 128;

// Whether P^T and dS^T have places of their own.
template <int HD> constexpr bool kEarly = HD == 64;

// DKV: of the kernel of dk and dv, which keeps queries' statistics too.
template <int HD, bool DKV> struct BackSizes {
    static constexpr int kBoxes = HD / 64;
    static constexpr int kOperand = kBoxes * kBox;            // bytes of a tile of Q, K, V or dO
    static constexpr int kStages = HD == 128 ? (DKV ? 4 : 5) : 8;
    static constexpr int kPlaces = DKV ? kStages / 2 + 1 : 0; // of the queries' lse and D
    // A tile's lse and D: planes of lse, of zeros and of D, of which a product's 16 more of K
    // are the first or the last two.  An infinite D so does not meet the scores.
    static constexpr int kFold = 3 * kFoldPlane;
    static constexpr int kOwn = !DKV && HD == 64 ? 2 : 1;     // places of the CTA's own Q and dO (or K and V), and of dq
    static constexpr int kBarriers = (DKV ? 11 : 7 + 4 * kOwn) + 2 * kStages;
    static constexpr int kSmem =
        1024 + (2 * kOwn + kStages) * kOperand + (kPlaces + (DKV ? 1 : 0)) * kFold + 8 * kBarriers + 32 + 4 * kValueWarps;
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

// A warp's columns from tensor memory, and its 16-bit P or dS to it.
__device__ __forceinline__ void load_columns(uint32_t addr, uint32_t (&v)[kCols]) {
    tmem_load32(addr, v);
    tmem_load_wait();
    tmem_loaded32(v);
}
template <class T> __device__ __forceinline__ void store_columns(uint32_t addr, const float (&v)[kCols]) {
    uint32_t w[kCols / 2];
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i) w[i] = pack_pair<T>(v[2 * i], v[2 * i + 1]);
    tmem_store16(addr, w);
    tmem_store_wait();
}
// 0 in the places whose bit is not set.
__device__ __forceinline__ void keep(float (&v)[kCols], uint32_t seen) {
#pragma unroll
    for (int i = 0; i < kCols; ++i)
        if (!(seen >> i & 1u)) v[i] = 0.f;
}
// What this warp read of tensor memory, or wrote to it, is behind it.
__device__ __forceinline__ void pass_on(uint32_t bar) {
    tcgen05_before_sync();
    __syncwarp();
    if (threadIdx.x % 32 == 0) mbar_arrive(bar);
}

template <class T, int HD>
__global__ void __launch_bounds__(kBackThreads, 1)
attention_dkv_kernel(const __grid_constant__ AttentionArgs a, const __grid_constant__ HeadMaps m,
                     const __grid_constant__ KeySplit split) {
    using Z = BackSizes<HD, true>;
    constexpr int ST = Z::kStages, SS = Z::kPlaces;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (1024 - (smem_addr(smem_raw) & 1023)) % 1024;
    const uint32_t k_at = smem_addr(smem), v_at = k_at + Z::kOperand, ring0 = k_at + 2 * Z::kOperand;
    uint8_t *ones = smem + (2 + ST) * Z::kOperand;            // the keys' side of lse, of D
    const uint32_t ones_at = smem_addr(ones), fold0 = ones_at + Z::kFold;
    uint64_t *bars = reinterpret_cast<uint64_t *>(ones + (1 + SS) * Z::kFold);
    const uint32_t kv_full = smem_addr(bars), full = kv_full + 8, empty = full + 8 * ST;
    const uint32_t s_full = empty + 8 * ST, dp_full = s_full + 8, p_ready = dp_full + 8, ds_ready = p_ready + 8;
    // where products are early: S and dP have been read, dS has been used
    const uint32_t s_taken = ds_ready + 8, dp_taken = s_taken + 8, ds_used = dp_taken + 8;
    const uint32_t done = ds_used + 8, drained = done + 8, unit_ready = drained + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + Z::kBarriers);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    uint32_t *bad_rows = tmem_slot + 4;                       // [warps of values]
    // fp16: dS's unit, the queries' largest sum |dO| and |D|, and the keys' |v|
    float *units = reinterpret_cast<float *>(bad_rows + kValueWarps);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (warp == kLoadWarp && lane == 0) {
        mbar_init(kv_full, 1);
        for (int s = 0; s < ST; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        mbar_init(s_full, 1);
        mbar_init(dp_full, 1);
        mbar_init(p_ready, kValueWarps);
        mbar_init(ds_ready, kValueWarps);
        mbar_init(s_taken, kValueWarps);
        mbar_init(dp_taken, kValueWarps);
        mbar_init(ds_used, 1);
        mbar_init(done, 1);
        mbar_init(drained, 1);
        mbar_init(unit_ready, 1);
        *abort = 0;
        fence_mbar_init();
        fence_async_shared();
    }
    if (warp == kTmemWarp) tmem_alloc<1>(smem_addr(tmem_slot), 512);
    if (threadIdx.x < 2 * kTile) {
        const int row = threadIdx.x % kTile, of_d = threadIdx.x / kTile;
        const uint32_t w0 = pack_pair<T>(fold_unit<T>(0), fold_unit<T>(1)), w1 = pack_pair<T>(fold_unit<T>(2), fold_unit<T>(3));
        *reinterpret_cast<uint4 *>(ones + 2 * of_d * kFoldPlane + fold_offset(row)) = make_uint4(w0, w1, 0, 0);
        if (of_d)
            for (int s = 0; s <= SS; ++s)                     // of the ones too
                *reinterpret_cast<uint4 *>(ones + s * Z::kFold + kFoldPlane + fold_offset(row)) = make_uint4(0, 0, 0, 0);
        fence_async_shared();
    }
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = *tmem_slot;
    grid_dependency();
    const AttentionWaiter wait{abort, m.timeouts};

    const int heads = a.batch * a.hkv;
    const int kh = int(blockIdx.x) % heads % a.hkv, b = int(blockIdx.x) % heads / a.hkv;
    const int unit = int(blockIdx.x) / heads, shared = split.first[split.tiles], shift = a.sk - a.sq;
    int tile = split.tiles + unit - shared;
    if (unit < shared)
        for (tile = 0; split.first[tile + 1] <= unit;) ++tile;
    const int k0 = tile * kTile;
    const QueryTiles tiles = query_tiles(a, k0);
    // pairs [begin, begin + total) of the tile's with each query tile of each head
    const int count = tiles.high - tiles.low, begin = unit < shared ? (unit - split.first[tile]) * split.chunk : 0;
    const int total = unit < shared ? min(split.chunk, count * a.group - begin) : count * a.group;
    // S^T, dP^T, P^T and dS^T, dv and dk; each warpgroup's P and dS at a step of its own
    const uint32_t p_at = kEarly<HD> ? tmem + 256 : tmem, ds_at = kEarly<HD> ? tmem + 320 : tmem + kTile;
    constexpr int kStep = kEarly<HD> ? kCols / 2 : kCols;
    const uint32_t dv_acc = tmem + 512 - 2 * HD, dk_acc = tmem + 512 - HD;

    if (warp == kLoadWarp) {                                  // loads
        if (total > 0) {
            if (elect_one()) {
                mbar_expect_tx(kv_full, 2 * Z::kOperand);
                for (int x = 0; x < Z::kBoxes; ++x) {
                    tma_load_4d(k_at + x * kBox, &m.k, 64 * x, k0, kh * m.k_head, b * m.k_batch, kv_full);
                    tma_load_4d(v_at + x * kBox, &m.v, 64 * x, k0, kh * m.v_head, b * m.v_batch, kv_full);
                }
            }
            __syncwarp();
            bool ok = true;
            uint32_t issued = 0;
            Turn<ST> ring;
            Turn<SS> place;
            for (int i = 0; i < total && ok; ++i) {
                const int h = kh * a.group + (begin + i) / count, q = (tiles.low + (begin + i) % count) * kTile;
                for (int x = 0; x < 2 && ok; ++x) {           // Q and its lse and D, dO
                    ok = __all_sync(0xffffffffu, wait(empty + 8 * ring.at, ring.turn ^ 1));
                    if (!ok) break;
                    if (elect_one()) {
                        const uint32_t to = ring0 + ring.at * Z::kOperand, bar = full + 8 * ring.at;
                        mbar_expect_tx(bar, Z::kOperand + (x == 0 ? 2 * kFoldPlane : 0));
                        for (int y = 0; y < Z::kBoxes; ++y)
                            tma_load_4d(to + y * kBox, x == 0 ? &m.q : &m.d_o, 64 * y, q, h * (x == 0 ? m.q_head : m.do_head),
                                        b * (x == 0 ? m.q_batch : m.do_batch), bar);
                        if (x == 0)
                            for (int y = 0; y < 2; ++y)
                                bulk_load(fold0 + place.at * Z::kFold + 2 * y * kFoldPlane,
                                          a.fold + ((int64_t(b) * a.hq + h) * a.sq_pad + q) * 16 + y * (kFoldPlane / 2), kFoldPlane, bar);
                    }
                    __syncwarp();
                    ring.next();
                    ++issued;
                }
                place.next();
            }
            // a CTA ends after its copies in flight, also where another warp gave up on them
            const uint32_t open = issued < uint32_t(ST) ? issued : ST;
            for (uint32_t i = issued - open; i < issued; ++i) wait(full + 8 * (i % ST), (i / ST) & 1, false);
            wait(kv_full, 0, false);
        }
    } else if (warp == kIssueWarp) {                          // products
        if (total > 0 && elect_one()) {
            const bool bf16 = std::is_same_v<T, __nv_bfloat16>;
            const int ksteps = (a.d + 15) / 16;
            const uint32_t is = mma_f16_desc(kTile, kTile, bf16, a.scale < 0.f, false);
            const uint32_t idp = mma_f16_desc(kTile, kTile, bf16, false, false);
            const uint32_t io = mma_f16_desc(kTile, ksteps * 16, bf16, false, true);
            Turn<ST> ring;
            bool ok = wait(kv_full, 0);
            // a 128 x 128 product over the head, S^T or dP^T, and over the 16 more of K
            auto across_head = [&](uint32_t d, uint32_t x, uint32_t y, uint32_t ones, uint32_t fold, uint32_t desc, uint32_t bar) {
                const uint64_t dx = desc_k_major(x), dy = desc_k_major(y);
                for (int k = 0; k < ksteps; ++k) {
                    const uint32_t at = (k / 4) * (kBox / 16) + (k % 4) * 2;
                    mma_f16(d, dx + at, dy + at, desc, k > 0);
                }
                mma_f16(d, desc_plain(ones, kFoldPlane, 128), desc_plain(fold, kFoldPlane, 128), desc, true);
                mma_commit<1>(bar);
            };
            // a product over the queries: P^T dO or dS^T Q
            auto across_queries = [&](uint32_t d, uint32_t x, uint32_t y, bool add) {
                const uint64_t dy = desc_k_across(y, kBox);
                for (int k = 0; k < kTile / 16; ++k)
                    mma_f16_tmem(d, x + (k / 2) * kStep + (k % 2) * 8, dy + k * (16 * 128 / 16), io, add || k > 0);
            };
            auto take = [&]() {
                ok = ok && wait(full + 8 * ring.at, ring.turn);
                const uint32_t at = ring.at;
                ring.next();
                return at;
            };
            uint32_t q = take(), o = take();
            Turn<SS> of_s, of_dp;                             // places of lse and D
            if (ok) {
                tcgen05_after_sync();
                across_head(tmem, k_at, ring0 + q * Z::kOperand, ones_at, fold0, is, s_full);
                across_head(tmem + kTile, v_at, ring0 + o * Z::kOperand, ones_at + kFoldPlane, fold0 + kFoldPlane, idp, dp_full);
            }
            for (int i = 0; i < total && ok; ++i) {
                const bool more = i + 1 < total;
                const uint32_t q_now = q, o_now = o;
                // the next pair's product, once its place is free
                auto next = [&](uint32_t &at, Turn<SS> &place, uint32_t d, uint32_t x, uint32_t plane, uint32_t desc, uint32_t bar,
                                uint32_t taken) {
                    if (!more) return;
                    at = take();
                    place.next();
                    if (kEarly<HD>) ok = ok && wait(taken, i & 1);
                    if (!ok) return;
                    tcgen05_after_sync();
                    across_head(d, x, ring0 + at * Z::kOperand, ones_at + plane, fold0 + place.at * Z::kFold + plane, desc, bar);
                };
                if (kEarly<HD>) next(q, of_s, tmem, k_at, 0, is, s_full, s_taken);
                ok = ok && wait(p_ready, i & 1);
                if (!ok) break;
                tcgen05_after_sync();
                across_queries(dv_acc, p_at, ring0 + o_now * Z::kOperand, i > 0);
                if (!kEarly<HD>) next(q, of_s, tmem, k_at, 0, is, s_full, s_taken);
                if (kEarly<HD>) next(o, of_dp, tmem + kTile, v_at, kFoldPlane, idp, dp_full, dp_taken);
                mma_commit<1>(empty + 8 * o_now);
                ok = ok && wait(ds_ready, i & 1);
                if (!ok) break;
                tcgen05_after_sync();
                across_queries(dk_acc, ds_at, ring0 + q_now * Z::kOperand, i > 0);
                if (kEarly<HD>) mma_commit<1>(ds_used);
                mma_commit<1>(empty + 8 * q_now);
                if (!kEarly<HD>) next(o, of_dp, tmem + kTile, v_at, kFoldPlane, idp, dp_full, dp_taken);
            }
            if (ok) mma_commit<1>(done);
            // nothing is in flight at the end
            mma_commit<1>(drained);
            wait(drained, 0, false);
        }
    } else if (kUnits<T> && warp == kTmemWarp) {              // the unit of dS
        if (total > 0) {
            float top = 0.f, sum = 0.f, most = 0.f;
            for (int i = lane; i < total; i += 32) {
                const int h = kh * a.group + (begin + i) / count, q = (tiles.low + (begin + i) % count) * kTile;
#pragma unroll
                for (int y = 0; y < kTile / 32; ++y) {
                    const float4 x = a.peak[((int64_t(b) * a.hq + h) * a.sq_pad + q) / 32 + y];
                    top = fmaxf(top, x.x);
                    sum = fmaxf(sum, x.y);
                    most = fmaxf(most, x.z);
                }
            }
            top = warp_max(top);
            sum = warp_max(sum);
            most = warp_max(most);
            if (lane == 0) {
                units[0] = unit_of(top);
                units[1] = sum;
                units[2] = most;
                mbar_arrive(unit_ready);
            }
            __syncwarp();
        }
    } else if (kUnits<T> && warp == kTmemWarp + 1) {          // the largest |v|
        if (total > 0) {
            const bool ok = __all_sync(0xffffffffu, wait(kv_full, 0));
            float top = 0.f;
            for (int x = lane; ok && x < Z::kOperand / 16; x += 32)
                top = fmaxf(top, finite_peak<T>(*reinterpret_cast<const uint4 *>(smem + Z::kOperand + 16 * x)));
            top = warp_max(top);
            if (lane == 0) {
                units[3] = top;
                a.v_peak[(int64_t(b) * a.hkv + kh) * ((a.sk + kTile - 1) / kTile) + tile] = top;
            }
            __syncwarp();
        }
        asm volatile("bar.arrive 1, %0;" ::"n"(32 * kValueWarps + 32) : "memory");
    } else if (warp < kValueWarps) {                          // values
        const int way = warp / 4, quarter = warp % 4, key = k0 + quarter * 32 + lane;
        const uint32_t lanes = uint32_t(quarter * 32) << 16;
        const uint32_t ts = tmem + lanes + kCols * way, tp = ts + kTile;
        const uint32_t to_p = p_at + lanes + kStep * way, to_ds = ds_at + lanes + kStep * way;
        const float c = score_scale(a.scale);
        const float2 c2 = make_float2(c, c);
        bool ok = true;
        float ds_unit = 1.f;                                  // dS is multiplied by it
        if (kUnits<T> && total > 0) {
            ok = __all_sync(0xffffffffu, wait(unit_ready, 0));
            ds_unit = units[0];
        }
        const float2 p2 = make_float2(kProbabilityExponent, kProbabilityExponent);
        const float2 unit2 = make_float2(ds_unit * kProbabilityUnit, ds_unit * kProbabilityUnit);
        const int k1 = k0 + kTile - 1, seen_by = last_position(a, key) - shift;
        int q0 = (tiles.low + (total > 0 ? begin % count : 0)) * kTile;
        for (int i = 0; i < total; ++i, q0 = q0 + kTile < tiles.high * kTile ? q0 + kTile : tiles.low * kTile) {
            ok = __all_sync(0xffffffffu, wait(s_full, i & 1));
            if (!ok) break;
            tcgen05_after_sync();
            // not all keys are seen by all queries, or some queries do not exist
            const bool masked = !(k1 <= q0 + shift && (k0 > q0 + kTile - 1 + shift - a.window || k1 < a.sinks)) || q0 + kTile > a.sq;
            uint32_t x[kCols], seen = 0xffffffffu;
            float p[kCols];
            load_columns(ts, x);
            if (kEarly<HD>) pass_on(s_taken);
#pragma unroll
            for (int e = 0; e < kCols; e += 2) {
                const float2 y = make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                const float2 f = kUnits<T> ? fma2(y, c2, p2) : mul2(y, c2);
                p[e] = exp2_fast(f.x);
                p[e + 1] = exp2_fast(f.y);
            }
            if (masked) {                                     // this warpgroup's columns that see the key
                const int at0 = q0 + kCols * way;
                seen = bits_to(seen_by - at0) & ~bits_to(key - shift - at0 - 1);
            }
            if (masked) keep(p, seen);
            if (kEarly<HD>) {
                // dP(i) is made after dv P(i - 1): P's place is free then
                ok = __all_sync(0xffffffffu, wait(dp_full, i & 1));
                if (!ok) break;
                tcgen05_after_sync();
            }
            store_columns<T>(to_p, p);
            pass_on(p_ready);
            if (!kEarly<HD>) {
                ok = __all_sync(0xffffffffu, wait(dp_full, i & 1));
                if (!ok) break;
                tcgen05_after_sync();
            }
            load_columns(tp, x);
            if (kEarly<HD>) pass_on(dp_taken);
#pragma unroll
            for (int e = 0; e < kCols; e += 2) {
                float2 f = mul2(make_float2(p[e], p[e + 1]), make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])));
                if constexpr (kUnits<T>) f = mul2(f, unit2);
                p[e] = f.x;
                p[e + 1] = f.y;
            }
            if (masked) keep(p, seen);                        // 0 times an infinity
            if (kEarly<HD> && i > 0) {
                ok = __all_sync(0xffffffffu, wait(ds_used, (i - 1) & 1));
                if (!ok) break;
                tcgen05_after_sync();
            }
            store_columns<T>(to_ds, p);
            pass_on(ds_ready);
        }
        if (total > 0) {
            ok = __all_sync(0xffffffffu, ok && wait(done, 0));
            tcgen05_after_sync();
        }
        // two warpgroups store dv, the others dk, every other 32 values of a row each
        float *part = nullptr;
        if (unit < shared)
            part = split.partial + ((int64_t(blockIdx.x) * 2 + way / 2) * kTile + quarter * 32 + lane) * HD;
        const bool exists = key < a.sk;
        const float f = way < 2 ? 1.f : a.scale, back = way < 2 ? kProbabilityUnit : over_unit(ds_unit);
        const uint32_t acc = (way < 2 ? dv_acc : dk_acc) + lanes;
        T *row = row_of<T>(way < 2 ? a.dv : a.dk, b, exists ? key : 0, kh);
        bool finite = true;
        for (int i = way % 2; i < (a.d + 31) / 32; i += 2) {
            uint32_t v[32];
            if (total == 0) {
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = 0u;
            } else if (ok) {
                tmem_load32(acc + 32 * i, v);
                tmem_load_wait();
                tmem_loaded32(v);
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = 0x7fffffffu;
            }
            if constexpr (kUnits<T>)
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * back);
            if (part != nullptr) {
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<uint4 *>(part + 32 * i + e) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                continue;
            }
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
                uint32_t w[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float u = __uint_as_float(v[e + 2 * y]) * f, z = __uint_as_float(v[e + 2 * y + 1]) * f;
                    if (32 * i + e < a.d) finite = finite && fabsf(u) < INFINITY && fabsf(z) < INFINITY;
                    w[y] = pack_pair<T>(u, z);
                }
                if (exists && 32 * i + e < a.d)
                    *reinterpret_cast<uint4 *>(row + 32 * i + e) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        // rows that are no numbers, again from the definition: dk and dv of a row together
        const uint32_t bad = __ballot_sync(0xffffffffu, ok && exists && !finite);
        if (lane == 0) bad_rows[warp] = bad;
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kValueWarps + (kUnits<T> ? 32 : 0)) : "memory");
        uint32_t again = bad_rows[quarter] | bad_rows[quarter + 4] | bad_rows[quarter + 8] | bad_rows[quarter + 12];
        if (again != 0 || unit < shared) {
            const bool past = kUnits<T> && total > 0 && past_half(ds_unit, units[1], units[3], units[2]);
            if (unit < shared && threadIdx.x == 0) split.past[blockIdx.x] = past;
            // a quarter's rows go round its warps
            for (int x = 0; again != 0; again &= again - 1, ++x)
                if (x % kWays == way) mend_dkv_row<T>(a, b, kh, k0, k0 + quarter * 32 + __ffs(int(again)) - 1, past);
        }
    }
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    if (warp == kTmemWarp) tmem_free<1>(tmem, 512);
}

// The tile of queries number w, the last queries of every head first.
struct QueryTile {
    int b, h, kh, q0;
    KeyTiles keys;
    __device__ __forceinline__ QueryTile(const AttentionArgs &a, int w) {
        const int heads = a.batch * a.hq;
        h = w % heads % a.hq;
        b = w % heads / a.hq;
        kh = h / a.group;
        q0 = (a.sq_pad / kTile - 1 - w / heads) * kTile;
        keys = key_tiles(a, q0);
    }
};

template <class T, int HD>
__global__ void __launch_bounds__(kBackThreads, 1)
attention_dq_kernel(const __grid_constant__ AttentionArgs a, const __grid_constant__ HeadMaps m, int items) {
    using Z = BackSizes<HD, false>;
    constexpr int ST = Z::kStages, OWN = Z::kOwn;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (1024 - (smem_addr(smem_raw) & 1023)) % 1024;
    const uint32_t own0 = smem_addr(smem), ring0 = own0 + 2 * OWN * Z::kOperand;      // [place][Q, dO]
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + (2 * OWN + ST) * Z::kOperand);
    const uint32_t qo_full = smem_addr(bars), qo_empty = qo_full + 8 * OWN, full = qo_empty + 8 * OWN, empty = full + 8 * ST;
    const uint32_t s_full = empty + 8 * ST, dp_full = s_full + 8, s_taken = dp_full + 8, dp_taken = s_taken + 8;
    const uint32_t ds_ready = dp_taken + 8, done = ds_ready + 16, dq_taken = done + 8 * OWN, drained = dq_taken + 8 * OWN;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + Z::kBarriers);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *bad_from = reinterpret_cast<int *>(tmem_slot + 2);   // the first round with rows that are no numbers
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rounds = (items + int(gridDim.x) - 1) / int(gridDim.x);

    if (warp == kLoadWarp && lane == 0) {
        for (int s = 0; s < OWN; ++s) {
            mbar_init(qo_full + 8 * s, 1);
            mbar_init(qo_empty + 8 * s, 1);
            mbar_init(done + 8 * s, 1);
            mbar_init(dq_taken + 8 * s, kValueWarps);
        }
        for (int s = 0; s < ST; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        mbar_init(s_full, 1);
        mbar_init(dp_full, 1);
        mbar_init(s_taken, kValueWarps);
        mbar_init(dp_taken, kValueWarps);
        // one for each place of dS: the next pair's can be complete before this one's is
        // asked for, and a barrier tells only two phases in a row apart
        mbar_init(ds_ready, kValueWarps);
        mbar_init(ds_ready + 8, kValueWarps);
        mbar_init(drained, 1);
        *abort = 0;
        *bad_from = rounds;
        fence_mbar_init();
        fence_async_shared();
    }
    if (warp == kTmemWarp) tmem_alloc<1>(smem_addr(tmem_slot), 512);
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = *tmem_slot;
    grid_dependency();
    const AttentionWaiter wait{abort, m.timeouts};
    const int shift = a.sk - a.sq;
    // S, dP, two places of dS (64 columns each), one of dq or two
    const uint32_t dq_acc = tmem + 384, ds_at = tmem + 256;

    if (warp == kLoadWarp) {                                  // loads
        bool ok = true;
        uint32_t issued = 0;
        Turn<ST> ring;
        Turn<OWN> own;
        uint32_t tiles = 0;
        for (int r = 0; r < rounds && ok; ++r) {
            const int w = item_of(r);
            if (w >= items) continue;
            const QueryTile t(a, w);
            if (t.keys.count() == 0) continue;
            ok = __all_sync(0xffffffffu, wait(qo_empty + 8 * own.at, own.turn ^ 1));
            if (!ok) break;
            if (elect_one()) {
                const uint32_t bar = qo_full + 8 * own.at, to = own0 + 2 * own.at * Z::kOperand;
                mbar_expect_tx(bar, 2 * Z::kOperand);
                for (int x = 0; x < Z::kBoxes; ++x) {
                    tma_load_4d(to + x * kBox, &m.q, 64 * x, t.q0, t.h * m.q_head, t.b * m.q_batch, bar);
                    tma_load_4d(to + Z::kOperand + x * kBox, &m.d_o, 64 * x, t.q0, t.h * m.do_head, t.b * m.do_batch, bar);
                }
            }
            __syncwarp();
            own.next();
            ++tiles;
            for (int j = t.keys.begin(); j < t.keys.high && ok; j = t.keys.next(j))
                for (int x = 0; x < 2 && ok; ++x) {           // K, V
                    ok = __all_sync(0xffffffffu, wait(empty + 8 * ring.at, ring.turn ^ 1));
                    if (!ok) break;
                    if (elect_one()) {
                        const uint32_t to = ring0 + ring.at * Z::kOperand, bar = full + 8 * ring.at;
                        mbar_expect_tx(bar, Z::kOperand);
                        for (int y = 0; y < Z::kBoxes; ++y)
                            tma_load_4d(to + y * kBox, x == 0 ? &m.k : &m.v, 64 * y, j * kTile,
                                        t.kh * (x == 0 ? m.k_head : m.v_head), t.b * (x == 0 ? m.k_batch : m.v_batch), bar);
                    }
                    __syncwarp();
                    ring.next();
                    ++issued;
                }
        }
        // a CTA ends after its copies in flight, also where another warp gave up on them
        const uint32_t open = issued < uint32_t(ST) ? issued : ST;
        for (uint32_t i = issued - open; i < issued; ++i) wait(full + 8 * (i % ST), (i / ST) & 1, false);
        const uint32_t open_own = tiles < uint32_t(OWN) ? tiles : OWN;
        for (uint32_t i = tiles - open_own; i < tiles; ++i) wait(qo_full + 8 * (i % OWN), (i / OWN) & 1, false);
    } else if (warp == kIssueWarp) {                          // products
        if (elect_one()) {
            const bool bf16 = std::is_same_v<T, __nv_bfloat16>;
            const int ksteps = (a.d + 15) / 16;
            const uint32_t is = mma_f16_desc(kTile, kTile, bf16, a.scale < 0.f, false);
            const uint32_t idp = mma_f16_desc(kTile, kTile, bf16, false, false);
            const uint32_t io = mma_f16_desc(kTile, ksteps * 16, bf16, false, true);
            Turn<ST> ring;
            bool ok = true;
            auto take = [&]() {
                ok = ok && wait(full + 8 * ring.at, ring.turn);
                const uint32_t at = ring.at;
                ring.next();
                return at;
            };
            auto across_head = [&](uint32_t d, uint32_t x, uint32_t y, uint32_t desc, uint32_t bar) {
                const uint64_t dx = desc_k_major(x), dy = desc_k_major(y);
                for (int k = 0; k < ksteps; ++k) {
                    const uint32_t at = (k / 4) * (kBox / 16) + (k % 4) * 2;
                    mma_f16(d, dx + at, dy + at, desc, k > 0);
                }
                mma_commit<1>(bar);
            };
            // A pair of tiles; the queries' keys are walked one tile of queries after the other.
            struct Step {
                bool there, first, last;
                uint32_t k_place;
                Turn<OWN> own;
            };
            int r = -1, j = 0, left = 0;
            KeyTiles keys = {0, 0, 0};
            Turn<OWN> own;
            auto advance = [&]() {
                Step s = {left > 0, false, false, 0, own};
                if (left > 0) {
                    j = keys.next(j);
                } else {
                    while (left == 0 && ++r < rounds) {
                        const int w = item_of(r);
                        if (w < items) keys = QueryTile(a, w).keys, left = keys.count();
                    }
                    if (left == 0) return s;
                    j = keys.begin();
                    s.there = s.first = true;
                }
                s.last = --left == 0;
                if (s.last) own.next();
                return s;
            };
            uint32_t made = 0, used = 0;                      // scores, products with dS
            // S and dP of a pair of tiles, each once its place has been read; V's place is
            // free then, and after a tile's last pair Q's and dO's
            auto scores = [&](Step &s) {
                if (s.first) ok = ok && wait(qo_full + 8 * s.own.at, s.own.turn);
                s.k_place = take();
                if (made > 0) ok = ok && wait(s_taken, (made - 1) & 1);
                if (!ok) return;
                tcgen05_after_sync();
                across_head(tmem, own0 + 2 * s.own.at * Z::kOperand, ring0 + s.k_place * Z::kOperand, is, s_full);
            };
            auto gradients = [&](const Step &s) {
                const uint32_t v_now = take();
                if (made > 0) ok = ok && wait(dp_taken, (made - 1) & 1);
                if (!ok) return;
                tcgen05_after_sync();
                across_head(tmem + kTile, own0 + (2 * s.own.at + 1) * Z::kOperand, ring0 + v_now * Z::kOperand, idp, dp_full);
                mma_commit<1>(empty + 8 * v_now);
                if (s.last) mma_commit<1>(qo_empty + 8 * s.own.at);
                ++made;
            };
            auto sum = [&](const Step &s) {
                if (s.first) ok = ok && wait(dq_taken + 8 * s.own.at, s.own.turn ^ 1);
                ok = ok && wait(ds_ready + 8 * (used & 1), (used >> 1) & 1);
                if (!ok) return;
                tcgen05_after_sync();
                const uint64_t dk = desc_k_across(ring0 + s.k_place * Z::kOperand, kBox);
                for (int k = 0; k < kTile / 16; ++k)
                    mma_f16_tmem(dq_acc + s.own.at * HD, ds_at + (used & 1) * 64 + 8 * k, dk + k * (16 * 128 / 16), io, !s.first || k > 0);
                mma_commit<1>(empty + 8 * s.k_place);
                if (s.last) mma_commit<1>(done + 8 * s.own.at);
                ++used;
            };
            // The next pair's S before this one's sum; dP as well for heads of 64, whose shorter
            // sum would wait for it less than it for the sum (all keys 1.69 ms, 1.78 the other
            // way round), and after it for heads of 128 (16384, window 4096: 2.42 ms for 2.66)
            constexpr bool BOTH = HD == 64;
            Step now = advance();
            if (now.there) scores(now);
            if (now.there && ok) gradients(now);
            while (now.there && ok) {
                Step next = advance();
                // a tile whose Q and dO come to these ones' place is waited for after this sum
                const bool early = next.there && (OWN > 1 || !next.first);
                if (early) scores(next);
                if (early && BOTH && ok) gradients(next);
                if (ok) sum(now);
                if (next.there && !early && ok) scores(next);
                if (next.there && !(early && BOTH) && ok) gradients(next);
                now = next;
            }
            // nothing is in flight at the end
            mma_commit<1>(drained);
            wait(drained, 0, false);
        }
    } else if (warp < kValueWarps) {                          // values
        const int way = warp / 4, quarter = warp % 4;
        const uint32_t lanes = uint32_t(quarter * 32) << 16;
        const uint32_t ts = tmem + lanes + kCols * way, tp = ts + kTile;
        const float c = score_scale(a.scale);
        bool ok = true;
        uint32_t i = 0;
        Turn<OWN> own;
        for (int r = 0; r < rounds; ++r) {
            const int w = item_of(r);
            if (w >= items) continue;
            const QueryTile t(a, w);
            const int row = t.q0 + quarter * 32 + lane, p = row + shift;
            const int p0 = t.q0 + shift, p1 = min(t.q0 + kTile, a.sq) - 1 + shift;
            const bool exists = row < a.sq;
            const float2 st = a.stats[(int64_t(t.b) * a.hq + t.h) * a.sq_pad + row];     // row < sq_pad
            const float unit = kUnits<T> ? a.unit[(int64_t(t.b) * a.hq + t.h) * a.sq_pad + row] : 1.f;
            const float lse = (kUnits<T> ? float(int(__float_as_uint(unit) >> 23) - 127) : 0.f) - st.x;     // of P in the unit
            const float2 c2 = make_float2(c, c), lse2 = make_float2(lse, lse), d2 = make_float2(-st.y, -st.y);
            for (int j = t.keys.begin(); j < t.keys.high && ok; j = t.keys.next(j), ++i) {
                ok = __all_sync(0xffffffffu, wait(s_full, i & 1));
                if (!ok) break;
                tcgen05_after_sync();
                const int k0 = j * kTile, k1 = k0 + kTile - 1, at0 = k0 + kCols * way;
                const bool masked = !(k1 <= p0 && (k0 > p1 - a.window || k1 < a.sinks));
                uint32_t x[kCols];
                float ds[kCols];
                load_columns(ts, x);
                pass_on(s_taken);
#pragma unroll
                for (int e = 0; e < kCols; e += 2) {
                    const float2 f = fma2(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), c2, lse2);
                    ds[e] = exp2_fast(f.x);
                    ds[e + 1] = exp2_fast(f.y);
                }
                ok = __all_sync(0xffffffffu, wait(dp_full, i & 1));
                if (!ok) break;
                tcgen05_after_sync();
                load_columns(tp, x);
                pass_on(dp_taken);
#pragma unroll
                for (int e = 0; e < kCols; e += 2) {
                    const float2 f = mul2(make_float2(ds[e], ds[e + 1]),
                                          add2(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), d2));
                    ds[e] = f.x;
                    ds[e + 1] = f.y;
                }
                if (masked) {
                    const uint32_t seen = bits_to(p - at0) & (~bits_to(p - a.window - at0) | bits_to(a.sinks - 1 - at0));
                    keep(ds, seen);
                }
                // the place's last product is done: dP(i) was issued after it
                store_columns<T>(ds_at + lanes + (i & 1) * 64 + kCols / 2 * way, ds);
                pass_on(ds_ready + 8 * (i & 1));
            }
            const bool some = t.keys.count() > 0;
            if (some) {
                ok = __all_sync(0xffffffffu, ok && wait(done + 8 * own.at, own.turn));
                tcgen05_after_sync();
            }
            // each warpgroup stores 32 values of a row
            T *to = row_of<T>(a.dq, t.b, exists ? row : 0, t.h);
            bool finite = true;
            uint32_t v[32];
            const bool mine = 32 * way < a.d;
            if (mine && some && ok) {
                tmem_load32(dq_acc + own.at * HD + lanes + 32 * way, v);
                tmem_load_wait();
                tmem_loaded32(v);
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = some ? 0x7fffffffu : 0u;
            }
            if (some) {
                pass_on(dq_taken + 8 * own.at);
                own.next();
            }
            if (!mine) continue;
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
                uint32_t o[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    float u = __uint_as_float(v[e + 2 * z]), g = __uint_as_float(v[e + 2 * z + 1]);
                    if constexpr (kUnits<T>) u *= over_unit(unit), g *= over_unit(unit);
                    u *= a.scale;
                    g *= a.scale;
                    if (32 * way + e < a.d) finite = finite && fabsf(u) < INFINITY && fabsf(g) < INFINITY;
                    o[z] = pack_pair<T>(u, g);
                }
                if (exists && 32 * way + e < a.d)
                    *reinterpret_cast<uint4 *>(to + 32 * way + e) = make_uint4(o[0], o[1], o[2], o[3]);
            }
            if (__any_sync(0xffffffffu, exists && !finite) && lane == 0) atomicMin(bad_from, r);
        }
        // rows that are no numbers, again from the definition
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kValueWarps) : "memory");
        for (int r = ok ? *bad_from : rounds; r < rounds; ++r) {
            const int w = item_of(r);
            if (w >= items) continue;
            const QueryTile t(a, w);
            const int row0 = t.q0 + quarter * 32, row = row0 + lane;
            // a quarter's rows go round its warps
            uint32_t again = __ballot_sync(0xffffffffu, lane % kWays == way && row < a.sq &&
                                                            any_in_row<T>(row_of<const T>(a.dq, t.b, row < a.sq ? row : 0, t.h), a.d));
            for (; again != 0; again &= again - 1) mend_dq_row<T>(a, t.b, t.h, t.q0, row0 + __ffs(int(again)) - 1);
        }
    }
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    if (warp == kTmemWarp) tmem_free<1>(tmem, 512);
}

// dv and dk of the shared tiles: a warp a row, four values a lane, the parts in their order.
template <class T, int HD>
__global__ void __launch_bounds__(256) key_join_kernel(const __grid_constant__ AttentionArgs a, const __grid_constant__ KeySplit split) {
    grid_dependency();
    const int heads = a.batch * a.hkv, lane = threadIdx.x % 32;
    const int64_t row = int64_t(blockIdx.x) * 8 + threadIdx.x / 32;
    const int at = int(row % kTile), head = int(row / kTile % heads), tile = int(row / kTile / heads), key = tile * kTile + at;
    if (key >= a.sk) return;
    const int kh = head % a.hkv, b = head / a.hkv;
    float g[2][4] = {};
    const bool mine = 4 * lane < HD;
    for (int p = split.first[tile]; p < split.first[tile + 1]; ++p)
#pragma unroll
        for (int x = 0; x < 2; ++x)
            if (mine) {
                const float4 v = *reinterpret_cast<const float4 *>(
                    split.partial + (((int64_t(p) * heads + head) * 2 + x) * kTile + at) * HD + 4 * lane);
                g[x][0] += v.x; g[x][1] += v.y; g[x][2] += v.z; g[x][3] += v.w;
            }
    bool finite = true;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const float f = x == 0 ? 1.f : a.scale;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            g[x][j] *= f;
            if (4 * lane < a.d) finite = finite && fabsf(g[x][j]) < INFINITY;
        }
        if (4 * lane < a.d)
            *reinterpret_cast<uint2 *>(row_of<T>(x == 0 ? a.dv : a.dk, b, key, kh) + 4 * lane) =
                make_uint2(pack_pair<T>(g[x][0], g[x][1]), pack_pair<T>(g[x][2], g[x][3]));
    }
    __syncwarp();                                             // after the stores above
    if (__all_sync(0xffffffffu, finite)) return;
    bool past = false;
    for (int p = split.first[tile]; p < split.first[tile + 1]; ++p)
        past = past || split.past[int64_t(p) * heads + head] != 0;
    mend_dkv_row<T>(a, b, kh, tile * kTile, key, past);
}

template <class T, int HD>
basp_status go(const AttentionArgs &a, const HeadMaps &m, const KeySplit &s, cudaStream_t stream) {
    constexpr auto dq = attention_dq_kernel<T, HD>;
    constexpr auto dkv = attention_dkv_kernel<T, HD>;
    constexpr size_t dq_smem = BackSizes<HD, false>::kSmem, dkv_smem = BackSizes<HD, true>::kSmem;
    if (!allow_shared_memory<dq, dq_smem>() || !allow_shared_memory<dkv, dkv_smem>()) return BASP_ERR_CUDA;
    const int64_t heads = int64_t(a.batch) * a.hkv, q = ceil_div(a.sq, kTile) * a.batch * a.hq;
    const int64_t k = (ceil_div(a.sk, kTile) - s.tiles + s.first[s.tiles]) * heads;
    if (q > kMaxSide - 1024 || k > kMaxSide) return BASP_ERR_TOO_LARGE;
    basp_status st = launch(dkv, dim3(unsigned(k)), dim3(kBackThreads), dkv_smem, 1, stream, a, m, s);
    if (st == BASP_OK && s.tiles > 0)
        st = launch(key_join_kernel<T, HD>, dim3(unsigned(s.tiles * heads * (kTile / 8))), dim3(256), 0, 1, stream, a, s);
    if (st != BASP_OK) return st;
    return launch(dq, dim3(unsigned(std::min<int64_t>(q, sm_count()))), dim3(kBackThreads), dq_smem, 1, stream, a, m, int(q));
}

}  // namespace

// A tile with more work than an SM has to do altogether (and than 64 pairs of tiles) is
// shared by CTAs of a quarter of that.  A shorter one is hidden behind the others, since the
// longest begin first: shared, those of 2 x 8192 x 32 heads of 64 with a window of 1024 took
// 641 us, not 630.
KeySplit key_split(const AttentionArgs &a) {
    KeySplit s = {};
    const int64_t tiles = ceil_div(a.sk, kTile), heads = int64_t(a.batch) * a.hkv;
    if (tiles > 65536) return s;                              // plenty of tiles, and a loop over them
    int64_t sum = 0;
    auto pairs = [&](int64_t t) {
        const QueryTiles q = query_tiles(a, int(t * kTile));
        return int64_t(q.high - q.low) * a.group;
    };
    for (int64_t t = 0; t < tiles; ++t) sum += pairs(t);
    const int64_t chunk = std::max<int64_t>(16, ceil_div(sum * heads, kSms * 4));
    if (chunk > (1 << 30)) return s;
    s.chunk = int(chunk);
    for (int64_t t = 0; t < tiles && s.tiles < kMostSplit; ++t) {
        const int64_t n = pairs(t);
        if (n <= 4 * chunk || s.first[s.tiles] + ceil_div(n, chunk) > 4096) break;
        s.first[s.tiles + 1] = s.first[s.tiles] + int(ceil_div(n, chunk));
        ++s.tiles;
    }
    return s;
}

int64_t key_split_parts(const AttentionArgs &a, const KeySplit &s) { return int64_t(s.first[s.tiles]) * a.batch * a.hkv; }

int64_t key_split_bytes(const AttentionArgs &a, const KeySplit &s) {
    return (ceil_div(key_split_parts(a, s), 4) * 4 + key_split_parts(a, s) * 2 * kTile * (a.d <= 64 ? 64 : 128)) * int64_t(sizeof(float));
}

basp_status launch_attention_backward(const AttentionArgs &a, const HeadMaps &m, const KeySplit &s, bool bf16,
                                      cudaStream_t stream) {
    if (bf16) return a.d <= 64 ? go<__nv_bfloat16, 64>(a, m, s, stream) : go<__nv_bfloat16, 128>(a, m, s, stream);
    return a.d <= 64 ? go<__half, 64>(a, m, s, stream) : go<__half, 128>(a, m, s, stream);
}

}  // namespace basp_fp8
