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
// A CTA has two tiles of 128 queries of a head.  Each has a warpgroup for its softmax,
// one query a thread, S and O in tensor memory (512 columns: 2 x 128 of S, 2 x up to 128
// of O); P takes the place of S as it is made, in the tensors' 16-bit type, and is the
// product's operand from there.  One thread issues all products, in the order
//     P0 V(j), S0(j + 1), P1 V(j), S1(j + 1),
// so that one tile's products run under the other's softmax; one warp loads K and V by
// TMA through a ring of tiles.  Keys are visited in tiles of 128; only tiles on the
// diagonal, at the window's far end and at the sinks' end look at each pair.
//
// A masked pair has P = 0, but 0 times an infinite or NaN value is NaN: a row that comes
// out so is computed again by its warp from the definition, which reads what the row
// sees alone.
#include <cuda.h>

#include "attention.cuh"
#include "attention_common.cuh"

namespace basp_fp8 {
namespace {

template <int HD> struct ForwardSizes {
    static constexpr int kBoxes = HD / 64;
    static constexpr int kOperand = kBoxes * kBox;            // bytes of a tile of Q, K or V
    static constexpr int kStages = HD == 128 ? 5 : 8;
    static constexpr int kBarriers = 1 + 2 * kStages + 7;
    static constexpr int kSmem = 1024 + (2 + kStages) * kOperand + 8 * kBarriers + 16;
    static constexpr int kO = 256;                            // O's tensor-memory columns begin here
};
// Three warpgroups, launched with 168 registers a thread: two softmaxes of 216, and 72
// for the warps that load and issue (256 x 216 + 128 x 72 = 384 x 168).
constexpr int kForwardThreads = 384;
constexpr int kSoftmaxRegisters = 216, kOtherRegisters = 72;
static_assert(256 * kSoftmaxRegisters + 128 * kOtherRegisters <= kForwardThreads * 168, "registers");

template <class T, int HD>
__global__ void __launch_bounds__(kForwardThreads, 1)
attention_forward_kernel(const __grid_constant__ AttentionArgs a, const __grid_constant__ HeadMaps m) {
    using Z = ForwardSizes<HD>;
    constexpr int ST = Z::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (1024 - (smem_addr(smem_raw) & 1023)) % 1024;
    const uint32_t q0 = smem_addr(smem), ring0 = q0 + 2 * Z::kOperand;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + (2 + ST) * Z::kOperand);
    const uint32_t q_full = smem_addr(bars), full = q_full + 8, empty = full + 8 * ST;
    const uint32_t s_full = empty + 8 * ST, p_full = s_full + 16, o_full = p_full + 16, drained = o_full + 16;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + Z::kBarriers);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (warp == 8 && lane == 0) {
        mbar_init(q_full, 1);
        for (int s = 0; s < ST; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full + 8 * t, 1);
            mbar_init(p_full + 8 * t, 4);
            mbar_init(o_full + 8 * t, 1);
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

    // The last queries, which have the most keys, first.
    const int heads = a.batch * a.hq, block = int(gridDim.x) / heads - 1 - int(blockIdx.x) / heads;
    const int h = int(blockIdx.x) % heads % a.hq, b = int(blockIdx.x) % heads / a.hq, kh = h / a.group;
    const int r0 = block * 2 * kTile;
    const KeyTiles tiles[2] = {key_tiles(a, r0), key_tiles(a, r0 + kTile)};
    // both tiles' keys: those of one that has any, or from the first one's first to the second one's last
    const KeyTiles &e0 = tiles[0].count() > 0 ? tiles[0] : tiles[1], &e1 = tiles[1].count() > 0 ? tiles[1] : e0;
    const KeyTiles all = {min(max(e0.first, e1.first), e0.low), e0.low, e1.high};

    if (warp >= 8) fewer_registers<kOtherRegisters>();
    if (warp == 8) {                                          // loads
        bool ok = true;
        uint32_t issued = 0;
        Turn<ST> ring;
        if (all.count() > 0) {
            if (elect_one()) {
                mbar_expect_tx(q_full, 2 * Z::kOperand);
                for (int t = 0; t < 2; ++t)
                    for (int x = 0; x < Z::kBoxes; ++x)
                        tma_load_4d(q0 + t * Z::kOperand + x * kBox, &m.q, 64 * x, r0 + t * kTile, h * m.q_head,
                                    b * m.q_batch, q_full);
            }
            __syncwarp();
            auto load = [&](const CUtensorMap *map, int j, int head, int batch) {
                ok = ok && __all_sync(0xffffffffu, wait(empty + 8 * ring.at, ring.turn ^ 1));
                if (!ok) return;
                if (elect_one()) {
                    mbar_expect_tx(full + 8 * ring.at, Z::kOperand);
                    for (int x = 0; x < Z::kBoxes; ++x)
                        tma_load_4d(ring0 + ring.at * Z::kOperand + x * kBox, map, 64 * x, j * kTile, head, batch,
                                    full + 8 * ring.at);
                }
                __syncwarp();
                ring.next();
                ++issued;
            };
            // in the order of use: K(0), V(0), K(1), V(1), ...
            for (int j = all.begin(); j < all.high && ok; j = all.next(j)) {
                load(&m.k, j, kh * m.k_head, b * m.k_batch);
                load(&m.v, j, kh * m.v_head, b * m.v_batch);
            }
            // a CTA ends after its copies in flight, also where another warp gave up on them
            const uint32_t open = issued < uint32_t(ST) ? issued : ST;
            for (uint32_t i = issued - open; i < issued; ++i) wait(full + 8 * (i % ST), (i / ST) & 1, false);
            wait(q_full, 0, false);
        }
    } else if (warp == 9) {                                   // products
        if (all.count() > 0 && elect_one()) {
            const bool bf16 = std::is_same_v<T, __nv_bfloat16>;
            const int ksteps = (a.d + 15) / 16;
            const uint32_t is = mma_f16_desc(kTile, kTile, bf16, a.scale < 0.f, false);
            const uint32_t io = mma_f16_desc(kTile, ksteps * 16, bf16, false, true);
            Turn<ST> ring;
            uint32_t p_turn[2] = {0, 0};
            bool some[2] = {false, false};                    // O has something to be added to
            bool ok = wait(q_full, 0);
            auto scores = [&](int t, uint32_t k_at) {
                const uint64_t dq = desc_k_major(q0 + t * Z::kOperand), dk = desc_k_major(ring0 + k_at * Z::kOperand);
                for (int k = 0; k < ksteps; ++k) {
                    const uint32_t at = (k / 4) * (kBox / 16) + (k % 4) * 2;
                    mma_f16(tmem + t * kTile, dq + at, dk + at, is, k > 0);
                }
                mma_commit<1>(s_full + 8 * t);
            };
            auto take = [&]() {                               // the ring's next tile, loaded
                ok = ok && wait(full + 8 * ring.at, ring.turn);
                const uint32_t at = ring.at;
                ring.next();
                return at;
            };
            int j = all.begin();
            uint32_t k_at = take();
            if (ok) {
                tcgen05_after_sync();
                for (int t = 0; t < 2; ++t)
                    if (tiles[t].has(j)) scores(t, k_at);
                mma_commit<1>(empty + 8 * k_at);
            }
            while (ok && j < all.high) {
                const int next = all.next(j);
                const uint32_t v_at = take();
                if (next < all.high) k_at = take();
                for (int t = 0; t < 2 && ok; ++t) {
                    if (tiles[t].has(j)) {
                        ok = wait(p_full + 8 * t, p_turn[t]);
                        if (!ok) break;
                        p_turn[t] ^= 1;
                        tcgen05_after_sync();
                        const uint64_t dv = desc_k_across(ring0 + v_at * Z::kOperand, kBox);
                        for (int k = 0; k < kTile / 16; ++k)
                            mma_f16_tmem(tmem + Z::kO + t * HD, tmem + t * kTile + 8 * k, dv + k * (16 * 128 / 16), io,
                                         some[t] || k > 0);
                        some[t] = true;
                        if (j + 1 == tiles[t].high) mma_commit<1>(o_full + 8 * t);
                    }
                    if (next < all.high && tiles[t].has(next)) scores(t, k_at);
                }
                if (!ok) break;
                mma_commit<1>(empty + 8 * v_at);
                if (next < all.high) mma_commit<1>(empty + 8 * k_at);
                j = next;
            }
            // nothing is in flight at the end
            mma_commit<1>(drained);
            wait(drained, 0, false);
        }
    } else if (warp < 8) {                                    // softmax
        more_registers<kSoftmaxRegisters>();
        const int t = warp / 4, quarter = warp % 4;
        const int row = r0 + t * kTile + quarter * 32 + lane, p = row + a.sk - a.sq;
        const int p0 = r0 + t * kTile + a.sk - a.sq, p1 = min(r0 + (t + 1) * kTile, a.sq) - 1 + a.sk - a.sq;
        const uint32_t lanes = uint32_t(quarter * 32) << 16;
        const uint32_t ts = tmem + lanes + t * kTile, to = tmem + lanes + Z::kO + t * HD;
        const float c = fmaxf(fabsf(a.scale) * kLog2e, 0x1p-126f);   // a scale of 0 leaves all scores alike
        const KeyTiles &mine = tiles[t];
        const int ochunks = (a.d + 31) / 32;
        float top = -INFINITY, l = 0.f;
        uint32_t turn = 0;
        bool ok = true, begun = false;
        for (int j = mine.begin(); j < mine.high; j = mine.next(j)) {
            ok = __all_sync(0xffffffffu, wait(s_full + 8 * t, turn));
            if (!ok) break;
            turn ^= 1;
            tcgen05_after_sync();
            uint32_t s[kTile];
#pragma unroll
            for (int i = 0; i < 4; ++i) tmem_load32(ts + 32 * i, s + 32 * i);
            tmem_load_wait();
#pragma unroll
            for (int i = 0; i < 4; ++i) tmem_loaded32(s + 32 * i);
            const int k0 = j * kTile, k1 = k0 + kTile - 1;
            if (!(k1 <= p0 && (k0 > p1 - a.window || k1 < a.sinks))) {      // not all rows see all keys
                const int last = p - k0, after = p - a.window - k0, sink = a.sinks - k0;
#pragma unroll
                for (int i = 0; i < kTile; ++i)
                    if (i > last || (i <= after && i >= sink)) s[i] = __float_as_uint(-INFINITY);
            }
            float high = fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
#pragma unroll
            for (int i = 2; i < kTile; i += 2)
                high = fmaxf(fmaxf(high, __uint_as_float(s[i])), __uint_as_float(s[i + 1]));
            high = fmaxf(high, top);
            if (!begun) {
                top = high;
                begun = true;
            } else {
                const bool grown = (high - top) * c > 8.f;
                if (__any_sync(0xffffffffu, grown)) {
                    const float f = grown ? exp2_fast((top - high) * c) : 1.f;
                    if (grown) top = high;
                    l *= f;
                    for (int i = 0; i < ochunks; ++i) {
                        uint32_t o[32];
                        tmem_load32(to + 32 * i, o);
                        tmem_load_wait();
                        tmem_loaded32(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_store32(to + 32 * i, o);
                    }
                }
            }
            const float shift = top == -INFINITY ? 0.f : -top * c;
            const float2 c2 = make_float2(c, c), shift2 = make_float2(shift, shift);
            float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t w[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int e = 64 * half + 2 * i;
                    float2 x = fma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2, shift2);
                    x.x = exp2_fast(x.x);
                    x.y = exp2_fast(x.y);
                    if (i % 2) sum1 = add2(sum1, x);
                    else sum0 = add2(sum0, x);
                    w[i] = pack_pair<T>(x.x, x.y);
                }
                tmem_store32(ts + 32 * half, w);
            }
            l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
            tmem_store_wait();
            tcgen05_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full + 8 * t);
        }
        if (mine.count() > 0) {
            ok = __all_sync(0xffffffffu, ok && wait(o_full + 8 * t, 0));
            tcgen05_after_sync();
        }
        const bool exists = row < a.sq, any = p >= 0;         // whoever sees anything sees itself
        const float inv = 1.f / l;
        bool finite = true;
        T *o_row = row_of<T>(a.o, b, exists ? row : 0, h);
        for (int i = 0; i < ochunks; ++i) {
            uint32_t o[32];
            if (ok && mine.count() > 0) {
                tmem_load32(to + 32 * i, o);
                tmem_load_wait();
                tmem_loaded32(o);
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0x7fffffffu;
            }
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
                uint32_t w[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float u = any ? __uint_as_float(o[e + 2 * x]) * inv : 0.f;
                    const float v = any ? __uint_as_float(o[e + 2 * x + 1]) * inv : 0.f;
                    if (32 * i + e < a.d) finite = finite && fabsf(u) < INFINITY && fabsf(v) < INFINITY;
                    w[x] = pack_pair<T>(u, v);
                }
                if (exists && 32 * i + e < a.d)
                    *reinterpret_cast<uint4 *>(o_row + 32 * i + e) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        if (exists && a.lse != nullptr)
            a.lse[(int64_t(b) * a.hq + h) * a.sq + row] =
                !any ? -INFINITY : ok ? top * fabsf(a.scale) + logf(l) : __uint_as_float(0x7fffffffu);
        // rows that are no numbers, again from the definition (Q's tile has been read)
        uint32_t again = __ballot_sync(0xffffffffu, ok && exists && !finite);
        float *scratch = reinterpret_cast<float *>(smem + t * Z::kOperand) + quarter * 2 * kMaxHeadDim;
        while (again != 0) {
            forward_row<T>(a, b, h, r0 + t * kTile + quarter * 32 + __ffs(int(again)) - 1, scratch);
            again &= again - 1;
        }
    }
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    if (warp == 10) tmem_free<1>(tmem, 512);
}

template <class T, int HD> basp_status go(const AttentionArgs &a, const HeadMaps &m, cudaStream_t stream) {
    constexpr auto kernel = attention_forward_kernel<T, HD>;
    if (!allow_shared_memory<kernel, ForwardSizes<HD>::kSmem>()) return BASP_ERR_CUDA;
    const int64_t ctas = ceil_div(a.sq, 2 * kTile) * a.batch * a.hq;
    return launch(kernel, dim3(unsigned(ctas)), dim3(kForwardThreads), ForwardSizes<HD>::kSmem, 1, stream, a, m);
}

}  // namespace

basp_status launch_attention_forward(const AttentionArgs &a, const HeadMaps &m, bool bf16, cudaStream_t stream) {
    if (bf16) return a.d <= 64 ? go<__nv_bfloat16, 64>(a, m, stream) : go<__nv_bfloat16, 128>(a, m, stream);
    return a.d <= 64 ? go<__half, 64>(a, m, stream) : go<__half, 128>(a, m, stream);
}

}  // namespace basp_fp8
