// attention_forward.cu -- attention with a window and sinks, forward, on the tensor
// cores.
//
// One pass over the keys that a tile of queries sees, with the running maximum m and
// sum l of its softmax:
//     S = Q K^T,  P = 2^(c S - c m),  l += rows of P,  O += P V,   o = O / l,
// c = |scale| log2(e); a negative scale negates Q inside the product.  m is raised only
// where a row's largest score has grown by more than 8 in the exponent of 2: P stays
// below 2^8, which 16 bits hold as exactly as values below 1, and O is hardly ever
// multiplied.
//
// A CTA has two tiles of 128 queries of a head at a time.  Each has a warpgroup for its
// softmax, one query a thread, S and O in tensor memory; P, in the tensors' 16-bit type,
// is the product's operand from there.  One thread issues all products, one warp loads K
// and V by TMA through a ring of tiles.  Keys are visited in tiles of 128; only tiles on
// the diagonal, at the window's far end and at the sinks' end look at each pair.
//
// Heads of 64 leave room in tensor memory for P beside S (2 x (128 of S + 64 of P + 64 of
// O) columns): S(j + 1) is made as soon as S(j) has been read, so that a softmax never
// waits for its scores.  Heads of 128 do not (2 x (128 + 128)): P takes the place of S,
// and one tile's products run under the other's softmax:
//     P0 V(j), S0(j + 1), P1 V(j), S1(j + 1).
//
// One CTA an SM walks the pairs of tiles with the grid's stride, those with the most keys
// first: the loads and first scores of the next pair run under the end of this one.
//
// A masked pair has P = 0, but 0 times an infinite or NaN value is NaN: where a row comes
// out so, and a value it does not see can be the reason, it is computed again by its warp
// from the definition, which reads what the row sees alone.
//
// 2 x 16384 x 16 heads of 128, window 4096: 645 us, 1.58 PFLOP/s of whole tiles, near what
// the tensor cores sustain under the power limit; 2 x 8192 x 32 heads of 64, window 1024:
// 195 us, 39 % of the tensor cores' cycles and as much of the exponentials': what bounds it is
// the chain from scores to P, with two warps for each scheduler.
#include <cuda.h>

#include <algorithm>

#include "attention.cuh"
#include "attention_common.cuh"

namespace basp_fp8 {
namespace {

template <int HD> struct ForwardSizes {
    static constexpr bool kEarly = HD == 64;                  // P has its own place
    static constexpr int kBoxes = HD / 64;
    static constexpr int kOperand = kBoxes * kBox;            // bytes of a tile of Q, K or V
    static constexpr int kStages = HD == 128 ? 5 : 8;
    static constexpr int kBarriers = 2 + 2 * kStages + 9;
    static constexpr int kSmem = 1024 + (2 + kStages) * kOperand + 8 * kBarriers + 16;
    // tensor-memory columns: S of the tiles, P, O
    static constexpr int kP = kEarly ? 256 : 0, kPStep = kEarly ? 64 : kTile;
    static constexpr int kO = kEarly ? 384 : 256;
};
// REST: what o loses in its rounding is stored too.  A kernel of its own, since the branch alone
// takes 195 us to 202 where it is not (2 x 8192 x 32 heads of 64, window 1024; 207 where it is).
//
// Three warpgroups, launched with 168 registers a thread: two softmaxes of 216, and 72
// for the warps that load and issue (256 x 216 + 128 x 72 = 384 x 168).
constexpr int kForwardThreads = 384;
constexpr int kSoftmaxRegisters = 216, kOtherRegisters = 72;
static_assert(256 * kSoftmaxRegisters + 128 * kOtherRegisters <= kForwardThreads * 168, "registers");

// The pair of tiles number w, the last queries of every head first.
struct Pair {
    int b, h, kh, r0;
    KeyTiles tiles[2], all;
    __device__ __forceinline__ Pair(const AttentionArgs &a, int w) {
        const int heads = a.batch * a.hq, blocks = (a.sq + 2 * kTile - 1) / (2 * kTile);
        h = w % heads % a.hq;
        b = w % heads / a.hq;
        kh = h / a.group;
        r0 = (blocks - 1 - w / heads) * 2 * kTile;
        tiles[0] = key_tiles(a, r0);
        tiles[1] = key_tiles(a, r0 + kTile);
        // both tiles' keys: those of one that has any, or from the first one's first to the second one's last
        const KeyTiles &e0 = tiles[0].count() > 0 ? tiles[0] : tiles[1], &e1 = tiles[1].count() > 0 ? tiles[1] : e0;
        all = {min(max(e0.first, e1.first), e0.low), e0.low, e1.high};
    }
};

template <class T, int HD, bool REST>
__global__ void __launch_bounds__(kForwardThreads, 1)
attention_forward_kernel(const __grid_constant__ AttentionArgs a, const __grid_constant__ HeadMaps m, int pairs) {
    using Z = ForwardSizes<HD>;
    constexpr int ST = Z::kStages;
    constexpr bool EARLY = Z::kEarly;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (1024 - (smem_addr(smem_raw) & 1023)) % 1024;
    const uint32_t q0 = smem_addr(smem), ring0 = q0 + 2 * Z::kOperand;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + (2 + ST) * Z::kOperand);
    const uint32_t q_full = smem_addr(bars), q_empty = q_full + 8, full = q_empty + 8, empty = full + 8 * ST;
    // of each tile: S is there, S has been read (EARLY), P is there, P V is done (EARLY: each, else the last)
    const uint32_t s_full = empty + 8 * ST, s_taken = s_full + 16, p_full = s_taken + 16, pv_done = p_full + 16;
    const uint32_t drained = pv_done + 16;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + Z::kBarriers);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (warp == 8 && lane == 0) {
        tma_prefetch_map(&m.q);
        tma_prefetch_map(&m.k);
        tma_prefetch_map(&m.v);
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int s = 0; s < ST; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full + 8 * t, 1);
            mbar_init(s_taken + 8 * t, 4);
            mbar_init(p_full + 8 * t, 4);
            mbar_init(pv_done + 8 * t, 1);
        }
        mbar_init(drained, 1);
        *abort = 0;
        fence_mbar_init();
        fence_async_shared();
    }
    if (warp == 10) tmem_alloc<1>(smem_addr(tmem_slot), 512);
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = *tmem_slot;
    grid_dependency();
    const AttentionWaiter wait{abort, m.timeouts};
    const int rounds = (pairs + int(gridDim.x) - 1) / int(gridDim.x);

    if (warp >= 8) fewer_registers<kOtherRegisters>();
    if (warp == 8) {                                          // loads
        bool ok = true;
        uint32_t issued = 0, turns = 0;
        Turn<ST> ring;
        for (int r = 0; r < rounds && ok; ++r) {
            const int w = item_of(r);
            if (w >= pairs) continue;
            const Pair p(a, w);
            if (p.all.count() == 0) continue;
            if (turns > 0) ok = __all_sync(0xffffffffu, wait(q_empty, (turns - 1) & 1));
            if (!ok) break;
            ++turns;
            if (elect_one()) {
                mbar_expect_tx(q_full, 2 * Z::kOperand);
                for (int t = 0; t < 2; ++t)
                    for (int x = 0; x < Z::kBoxes; ++x)
                        tma_load_4d(q0 + t * Z::kOperand + x * kBox, &m.q, 64 * x, p.r0 + t * kTile, p.h * m.q_head,
                                    p.b * m.q_batch, q_full);
            }
            __syncwarp();
            auto load = [&](bool value, int j) {
                ok = ok && __all_sync(0xffffffffu, wait(empty + 8 * ring.at, ring.turn ^ 1));
                if (!ok) return;
                if (elect_one()) {
                    mbar_expect_tx(full + 8 * ring.at, Z::kOperand);
                    for (int x = 0; x < Z::kBoxes; ++x)
                        tma_load_4d(ring0 + ring.at * Z::kOperand + x * kBox, value ? &m.v : &m.k, 64 * x, j * kTile,
                                    p.kh * (value ? m.v_head : m.k_head), p.b * (value ? m.v_batch : m.k_batch),
                                    full + 8 * ring.at);
                }
                __syncwarp();
                ring.next();
                ++issued;
            };
            // in the order of use
            load(false, p.all.begin());
            for (int j = p.all.begin(); j < p.all.high && ok;) {
                const int next = p.all.next(j);
                if (EARLY && next < p.all.high) load(false, next);
                load(true, j);
                if (!EARLY && next < p.all.high) load(false, next);
                j = next;
            }
        }
        // a CTA ends after its copies in flight, also where another warp gave up on them
        const uint32_t open = issued < uint32_t(ST) ? issued : ST;
        for (uint32_t i = issued - open; i < issued; ++i) wait(full + 8 * (i % ST), (i / ST) & 1, false);
        if (turns > 0) wait(q_full, (turns - 1) & 1, false);
    } else if (warp == 9) {                                   // products
        if (elect_one()) {
            const bool bf16 = std::is_same_v<T, __nv_bfloat16>;
            const int ksteps = (a.d + 15) / 16;
            const uint32_t is = mma_f16_desc(kTile, kTile, bf16, a.scale < 0.f, false);
            const uint32_t io = mma_f16_desc(kTile, ksteps * 16, bf16, false, true);
            Turn<ST> ring;
            uint32_t turns = 0, made[2] = {0, 0}, used[2] = {0, 0};   // S and P of each tile
            bool ok = true;
            auto take = [&]() {                               // the ring's next tile, loaded
                ok = ok && wait(full + 8 * ring.at, ring.turn);
                const uint32_t at = ring.at;
                ring.next();
                return at;
            };
            auto scores = [&](int t, uint32_t k_at) {
                if (EARLY && made[t] > 0) ok = ok && wait(s_taken + 8 * t, (made[t] - 1) & 1);
                if (!ok) return;
                ++made[t];
                tcgen05_after_sync();
                const uint64_t dq = desc_k_major(q0 + t * Z::kOperand), dk = desc_k_major(ring0 + k_at * Z::kOperand);
                for (int k = 0; k < ksteps; ++k) {
                    const uint32_t at = (k / 4) * (kBox / 16) + (k % 4) * 2;
                    mma_f16(tmem + t * kTile, dq + at, dk + at, is, k > 0);
                }
                mma_commit<1>(s_full + 8 * t);
            };
            for (int r = 0; r < rounds && ok; ++r) {
                const int w = item_of(r);
                if (w >= pairs) continue;
                const Pair p(a, w);
                if (p.all.count() == 0) continue;
                bool some[2] = {false, false};                // O has something to be added to
                ok = wait(q_full, turns & 1);
                ++turns;
                int j = p.all.begin();
                uint32_t k_at = take();
                if (!ok) break;
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    if (p.tiles[t].has(j)) scores(t, k_at);
                if (!ok) break;
                mma_commit<1>(empty + 8 * k_at);
                if (p.all.next(j) >= p.all.high) mma_commit<1>(q_empty);
                auto values = [&](int t, uint32_t v_at) {
                    ok = ok && wait(p_full + 8 * t, used[t] & 1);
                    if (!ok) return;
                    ++used[t];
                    tcgen05_after_sync();
                    const uint64_t dv = desc_k_across(ring0 + v_at * Z::kOperand, kBox);
                    for (int k = 0; k < kTile / 16; ++k)
                        mma_f16_tmem(tmem + Z::kO + t * HD, tmem + Z::kP + t * Z::kPStep + 8 * k, dv + k * (16 * 128 / 16), io,
                                     some[t] || k > 0);
                    some[t] = true;
                    if (EARLY || j + 1 == p.tiles[t].high) mma_commit<1>(pv_done + 8 * t);
                };
                while (j < p.all.high) {
                    const int next = p.all.next(j);
                    const bool more = next < p.all.high, last = more && p.all.next(next) >= p.all.high;
                    if constexpr (EARLY) {
                        if (more) {
                            k_at = take();
#pragma unroll
                            for (int t = 0; t < 2; ++t)
                                if (p.tiles[t].has(next)) scores(t, k_at);
                            if (!ok) break;
                            mma_commit<1>(empty + 8 * k_at);
                            if (last) mma_commit<1>(q_empty);
                        }
                        const uint32_t v_at = take();
#pragma unroll
                        for (int t = 0; t < 2; ++t)
                            if (p.tiles[t].has(j)) values(t, v_at);
                        if (!ok) break;
                        mma_commit<1>(empty + 8 * v_at);
                    } else {
                        const uint32_t v_at = take();
                        if (more) k_at = take();
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (p.tiles[t].has(j)) values(t, v_at);
                            if (more && p.tiles[t].has(next)) scores(t, k_at);
                        }
                        if (!ok) break;
                        mma_commit<1>(empty + 8 * v_at);
                        if (more) mma_commit<1>(empty + 8 * k_at);
                        if (last) mma_commit<1>(q_empty);
                    }
                    j = next;
                }
            }
            // nothing is in flight at the end
            mma_commit<1>(drained);
            wait(drained, 0, false);
        }
    } else if (warp < 8) {                                    // softmax
        more_registers<kSoftmaxRegisters>();
        const int t = warp / 4, quarter = warp % 4;
        const uint32_t lanes = uint32_t(quarter * 32) << 16;
        const uint32_t ts = tmem + lanes + t * kTile, tp = tmem + lanes + Z::kP + t * Z::kPStep;
        const uint32_t to = tmem + lanes + Z::kO + t * HD;
        const float c = fmaxf(fabsf(a.scale) * kLog2e, 0x1p-126f);   // a scale of 0 leaves all scores alike
        const int ochunks = (a.d + 31) / 32;
        uint32_t n = 0, sums = 0;                             // tiles of keys, pairs of tiles with any
        int bad_from = rounds;                                // the first round with rows that are no numbers
        bool ok = true;
        for (int r = 0; r < rounds; ++r) {
            const int w = item_of(r);
            if (w >= pairs) continue;
            int b, h, row0;
            KeyTiles mine;
            {
                const Pair p(a, w);
                b = p.b;
                h = p.h;
                row0 = p.r0 + t * kTile;
                mine = t == 0 ? p.tiles[0] : p.tiles[1];
            }
            const int row = row0 + quarter * 32 + lane, p = row + a.sk - a.sq;
            const int p0 = row0 + a.sk - a.sq, p1 = min(row0 + kTile, a.sq) - 1 + a.sk - a.sq;
            float top = -INFINITY, l = 0.f;
            bool begun = false;
            for (int j = mine.begin(); j < mine.high && ok; j = mine.next(j), ++n) {
                ok = __all_sync(0xffffffffu, wait(s_full + 8 * t, n & 1));
                if (!ok) break;
                tcgen05_after_sync();
                uint32_t s[kTile];
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_load32(ts + 32 * i, s + 32 * i);
                tmem_load_wait();
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_loaded32(s + 32 * i);
                if constexpr (EARLY) {
                    tcgen05_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_taken + 8 * t);
                }
                const int k0 = j * kTile, k1 = k0 + kTile - 1;
                if (!(k1 <= p0 && (k0 > p1 - a.window || k1 < a.sinks))) {      // not all rows see all keys
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int at = k0 + 32 * i;
                        const uint32_t seen = bits_to(p - at) & (~bits_to(p - a.window - at) | bits_to(a.sinks - 1 - at));
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(seen >> e & 1u)) s[32 * i + e] = __float_as_uint(-INFINITY);
                    }
                }
                float high[4] = {top, top, top, top};
#pragma unroll
                for (int i = 0; i < kTile; i += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        high[e] = max3(high[e], __uint_as_float(s[i + 2 * e]), __uint_as_float(s[i + 2 * e + 1]));
                high[0] = fmaxf(fmaxf(high[0], high[1]), fmaxf(high[2], high[3]));
                const bool grown = !begun || (high[0] - top) * c > 8.f;
                const bool again = __any_sync(0xffffffffu, begun && grown);      // O is multiplied
                const float f = grown ? exp2_fast((top - high[0]) * c) : 1.f;
                if (grown) top = high[0];
                if (again) l *= f;
                begun = true;
                const float shift = top == -INFINITY ? 0.f : -top * c;
                const float2 c2 = make_float2(c, c), shift2 = make_float2(shift, shift);
                float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
                // P takes the place of S in registers too, until its place in tensor memory is free
#pragma unroll
                for (int i = 0; i < kTile / 2; ++i) {
                    float2 x = fma2(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), c2, shift2);
                    x.x = exp2_fast(x.x);
                    x.y = exp2_fast(x.y);
                    if (i % 2) sum1 = add2(sum1, x);
                    else sum0 = add2(sum0, x);
                    s[i] = pack_pair<T>(x.x, x.y);
                }
                if constexpr (EARLY) {                        // P's place and O are free
                    if (n > 0) ok = __all_sync(0xffffffffu, wait(pv_done + 8 * t, (n - 1) & 1));
                    if (!ok) break;
                    tcgen05_after_sync();
                }
                if (again)
                    for (int i = 0; i < ochunks; ++i) {
                        uint32_t o[32];
                        tmem_load32(to + 32 * i, o);
                        tmem_load_wait();
                        tmem_loaded32(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_store32(to + 32 * i, o);
                    }
                tmem_store32(tp, s);
                tmem_store32(tp + 32, s + 32);
                l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
                tmem_store_wait();
                tcgen05_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * t);
            }
            const bool some = mine.count() > 0;
            if (some) {
                ok = __all_sync(0xffffffffu, ok && wait(pv_done + 8 * t, EARLY ? (n - 1) & 1 : sums & 1));
                tcgen05_after_sync();
                ++sums;
            }
            const bool exists = row < a.sq, any = p >= 0;     // whoever sees anything sees itself
            const float inv = 1.f / l;
            bool finite = true;
            T *o_row = row_of<T>(a.o, b, exists ? row : 0, h);
            int8_t *rest_row = REST ? row_of<int8_t>(a.rest, b, exists ? row : 0, h) : nullptr;
            const bool rest16 = REST && (uintptr_t(a.rest.p) | uint64_t(a.rest.sb | a.rest.ss | a.rest.sh)) % 16 == 0;
            for (int i = 0; i < ochunks; ++i) {
                uint32_t o[32], lost[8];
                if (ok && some) {
                    tmem_load32(to + 32 * i, o);
                    tmem_load_wait();
                    tmem_loaded32(o);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0x7fffffffu;
                }
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    uint32_t v[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float y = any ? __uint_as_float(o[e + 2 * x]) * inv : 0.f;
                        const float z = any ? __uint_as_float(o[e + 2 * x + 1]) * inv : 0.f;
                        if (32 * i + e < a.d) finite = finite && fabsf(y) < INFINITY && fabsf(z) < INFINITY;
                        v[x] = pack_pair<T>(y, z);
                    }
                    if (exists && 32 * i + e < a.d)
                        *reinterpret_cast<uint4 *>(o_row + 32 * i + e) = make_uint4(v[0], v[1], v[2], v[3]);
                    if constexpr (REST) {
                        int x[8];
#pragma unroll
                        for (int y = 0; y < 8; ++y) {
                            const float2 r = unpack_pair<T>(v[y / 2]);
                            x[y] = lost_of<T>(any ? __uint_as_float(o[e + y]) * inv : 0.f, y % 2 ? r.y : r.x);
                        }
                        lost[e / 4] = lost_bytes(x[0], x[1], x[2], x[3]);
                        lost[e / 4 + 1] = lost_bytes(x[4], x[5], x[6], x[7]);
                    }
                }
                if constexpr (REST)                           // 16 bytes at a time where that can be
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int at = 32 * i + 16 * x;
                        if (!exists) continue;
                        if (rest16 && at + 16 <= a.d) {
                            *reinterpret_cast<uint4 *>(rest_row + at) = make_uint4(lost[4 * x], lost[4 * x + 1], lost[4 * x + 2], lost[4 * x + 3]);
                        } else {
                            if (at < a.d) *reinterpret_cast<uint2 *>(rest_row + at) = make_uint2(lost[4 * x], lost[4 * x + 1]);
                            if (at + 8 < a.d) *reinterpret_cast<uint2 *>(rest_row + at + 8) = make_uint2(lost[4 * x + 2], lost[4 * x + 3]);
                        }
                    }
            }
            if (exists && a.lse != nullptr)
                a.lse[(int64_t(b) * a.hq + h) * a.sq + row] =
                    !any ? -INFINITY : ok ? top * fabsf(a.scale) + logf(l) : __uint_as_float(0x7fffffffu);
            if (bad_from == rounds && __any_sync(0xffffffffu, exists && !finite)) bad_from = r;
        }
        // Rows that are no numbers, again from the definition; at the end, since the CTA's
        // other warps would wait for them.
        for (int r = ok ? bad_from : rounds; r < rounds; ++r) {
            const int w = item_of(r);
            if (w >= pairs) continue;
            const Pair p(a, w);
            const int row0 = p.r0 + t * kTile, row = row0 + quarter * 32 + lane;
            uint32_t again = __ballot_sync(0xffffffffu, row < a.sq && any_in_row<T>(row_of<const T>(a.o, p.b, row < a.sq ? row : 0, p.h), a.d));
            for (; again != 0; again &= again - 1) {
                const int i = row0 + quarter * 32 + __ffs(int(again)) - 1;
                if (masked_keys_not_finite<T>(a, a.v, p.b, p.kh, row0, i + a.sk - a.sq)) forward_row<T, false>(a, p.b, p.h, i);
            }
        }
    }
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    if (warp == 10) tmem_free<1>(tmem, 512);
}

template <class T, int HD, bool REST> basp_status go_for(const AttentionArgs &a, const HeadMaps &m, cudaStream_t stream) {
    constexpr auto kernel = attention_forward_kernel<T, HD, REST>;
    if (!allow_shared_memory<kernel, ForwardSizes<HD>::kSmem>()) return BASP_ERR_CUDA;
    const int64_t pairs = ceil_div(a.sq, 2 * kTile) * a.batch * a.hq;
    if (pairs > kMaxSide - 1024) return BASP_ERR_TOO_LARGE;
    const int64_t ctas = std::min<int64_t>(pairs, sm_count());
    return launch(kernel, dim3(unsigned(ctas)), dim3(kForwardThreads), ForwardSizes<HD>::kSmem, 1, stream, a, m, int(pairs));
}

template <class T, int HD> basp_status go(const AttentionArgs &a, const HeadMaps &m, cudaStream_t stream) {
    return a.rest.p != nullptr ? go_for<T, HD, true>(a, m, stream) : go_for<T, HD, false>(a, m, stream);
}

}  // namespace

basp_status launch_attention_forward(const AttentionArgs &a, const HeadMaps &m, bool bf16, cudaStream_t stream) {
    if (bf16) return a.d <= 64 ? go<__nv_bfloat16, 64>(a, m, stream) : go<__nv_bfloat16, 128>(a, m, stream);
    return a.d <= 64 ? go<__half, 64>(a, m, stream) : go<__half, 128>(a, m, stream);
}

}  // namespace basp_fp8
