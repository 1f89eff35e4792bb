// Attention of a few drafted tokens over a paged cache:
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q.k_t - max),
// over the places t < ctx of a sequence and the drafts j whose bit the row's
// mask has.
//
// The rows of a tile are (token, head of a key head's group) pairs, 16 of them:
// one m16 tile of mma.sync, so every key and value is read once for all of
// them.  Work is counted in units of 16 cached tokens over all (sequence, key
// head, tile) segments and dealt to the blocks in equal shares, whatever the
// sequences' lengths; a block walks its share segment by segment.  In a
// block, each warp takes every eighth unit with a ring of its own: a lane
// orders the unit's keys and values from the tensor map (16 tokens are always
// in one page), two to five units ahead, and the warp multiplies, takes
// the softmax with a running maximum and sum, and multiplies again, without a
// barrier to other warps until the segment ends.  Then the warps' results are
// joined in shared memory; a segment that several blocks share is joined by
// the second launch (attn_join_kernel) in the order of its pieces, so no
// result depends on timing.
//
// Precision: products of 16-bit numbers in fp32 sums; probabilities enter the
// second product in the values' 16-bit type (bf16 for INT8 codes, which are
// exact in 16 bits: a key's scale multiplies its score, a value's scale its
// probability, and no range of the scales is lost), fp16 ones times 2^15
// (prob_lift).  They have parts of 11 or 8 bits, so many that the output's own
// rounding is what is left of their error: two, three of bf16 for an fp32 output, one
// of fp16 for a bf16 output.  With one part of as many bits as the output a place
// that has most of the weight moves all values of a row the same way: errors 1.3 to
// 1.5 times those of the rounded definition, where they are now the same.  One
// part would take 64 streams of D 64, 128, 256 in 70, 102, 113 us instead of 73, 103, 129,
// 8 x 64 drafts in 52 instead of 60, 5 drafts over 120001 INT8 places in 38 instead of 41.
//
// One token over 131071 bf16 places (4 key heads of 128): 49 to 50 us, 5.4 TB/s; the stream itself runs at 7.1 TB/s for 38 us,
// between 5 us of start (lengths, page, first copies) and 4 of joining.  1000 places: 8.4 us.  64 streams of 400 to 8190
// places: 103 us (565 MB).  INT8 codes cost instructions to widen: 14 rows over 65536 places (69 MB) 34 us, 7 rows 33, bf16
// (134 MB) 30.
#include <atomic>

#include "attn_tree.cuh"

namespace w4k {
namespace {

template <int D, int CT>
struct At {
    static constexpr int kEb = CT == T_I8 ? 1 : 2;
    static constexpr int kRow = D * kEb;                      // bytes of a token
    static constexpr int kBox = kRow < 128 ? kRow : 128;      // bytes of a box row
    static constexpr int kBoxes = kRow / kBox;
    static constexpr int kHalf = kAtUnit * kRow;              // a unit's keys (or values)
    static constexpr int kSlot = 2 * kHalf;
    // (two blocks of four warps per SM: 1 token over 131071 places 52.1 us, one of eight 48.7; 64 streams the same)
    static constexpr int kWarps = D == 256 ? 4 : 8;
    static constexpr int kParts = kWarps == 4 ? 1 : 2;        // joined row blocks: warps take turns on one
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kRing = 192 * 1024 / (kWarps * kSlot);
    static constexpr int kSlots = kRing > 6 ? 6 : kRing;      // units ahead of a warp
    static constexpr int kPad = D + 8;                        // floats of a joined row: rows spread over the banks
    // shared memory
    static constexpr int oRing = 0;
    static_assert(kWarps * kAtRows * kPad * 4 <= kWarps * kSlots * kSlot, "the rings hold every warp's result");
    static constexpr int oJoin = kWarps * kSlots * kSlot;                              // [kParts][16][kPad]
    static constexpr int oScale = oJoin + kParts * kAtRows * kPad * 4;             // [warps][slots][2][16]
    static constexpr int oMl = oScale + (CT == T_I8 ? kWarps * kSlots * 2 * kAtUnit * 4 : 0);   // [warps][2][16]
    static constexpr int oFin = oMl + kWarps * 2 * kAtRows * 4;                        // [2][16]
    static constexpr int oBars = oFin + 2 * kAtRows * 4;
    static constexpr int oOk = oBars + kWarps * kSlots * 8;                            // [warps][slots]: the page is there
    static constexpr int oWarpSum = (oOk + kWarps * kSlots * 4 + 7) / 8 * 8;
    static constexpr int oPre = oWarpSum + kWarps * 4;
    static constexpr int smem(int B) { return oPre + (B + 1) * 4 + 1024; }              // and the alignment of the ring
    static_assert(kSlots >= 2, "two units per warp");
    static_assert(oPre + (kAtMaxSeq + 1) * 4 + 1024 <= 232448, "shared memory of a block");
};

// The byte at column x of token t in a half slot, as the copies with a swizzle lay it.
template <int D, int CT>
__device__ __forceinline__ uint32_t place_of(int t, int x)
{
    using C = At<D, CT>;
    if constexpr (C::kBox == 128) {
        const int o = t * 128 + (x & 127);
        return static_cast<uint32_t>((x >> 7) * (kAtUnit * 128) + (o ^ ((t & 7) << 4)));
    } else {                                                  // 64-byte rows: two tokens to 128 bytes
        const int o = t * 64 + x;
        return static_cast<uint32_t>(o ^ ((o >> 7 & 3) << 4));
    }
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// c += a b, 16 x 8 x 16, fp16 or bf16 operands.
template <int T>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (T == T_F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int T>
__device__ __forceinline__ void codes16(uint32_t c, uint32_t& h01, uint32_t& h23)
{
    if constexpr (T == T_F16) i8_to_f16(c, h01, h23);
    else i8_to_bf16(c, h01, h23);
}

// kAdd: a unit's products are added to the output in fp32.
template <int D, int CT, int QT, int kParts, bool kAdd>
__global__ void __launch_bounds__(At<D, CT>::kThreads, 1) attn_tree_kernel(const __grid_constant__ AttnArgs A)
{
    using C = At<D, CT>;
    constexpr int PT = CT == T_F16 ? T_F16 : T_BF16;          // type of the second product
    constexpr int W = C::kWarps;
    constexpr float kLift = prob_lift(PT, 0.0f);
    extern __shared__ uint8_t raw[];
    uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    float* join_s = reinterpret_cast<float*>(smem + C::oJoin);
    float* ml_s = reinterpret_cast<float*>(smem + C::oMl);
    float* fin_s = reinterpret_cast<float*>(smem + C::oFin);
    volatile int* ok_s = reinterpret_cast<volatile int*>(smem + C::oOk) + warp * C::kSlots;
    int* pre_s = reinterpret_cast<int*>(smem + C::oPre);
    const uint32_t bars = smem_u32(smem + C::oBars) + static_cast<uint32_t>(warp * C::kSlots * 8);
    uint8_t* ring = smem + C::oRing + warp * C::kSlots * C::kSlot;
    const uint32_t ring_a = smem_u32(ring);
    float* scale_s = reinterpret_cast<float*>(smem + C::oScale) + warp * C::kSlots * 2 * kAtUnit;

    if (lane == 0) {
        if (warp == 0) {
            prefetch_map(&A.kmap);
            prefetch_map(&A.vmap);
        }
        for (int k = 0; k < C::kSlots; ++k) mbar_init(bars + 8 * k, 1);
        fence_mbar_init();
    }
    __syncwarp();
    pdl_wait();
    pdl_launch_dependents();                    // (behind the wait: the joining launch reads this one's inputs early)
    const Layout lay = block_layout<C::kThreads>(A, kAtRows, kAtUnit, pre_s, reinterpret_cast<int*>(smem + C::oWarpSum));
    if (blockIdx.x == 0 && A.b.B > 32)          // for the joining launch
        for (int b = tid; b <= A.b.B; b += C::kThreads) A.head[b] = pre_s[b];
    const int2 range = block_units(lay, A, static_cast<int>(blockIdx.x), kAtUnit);
    const int us = range.x, ue = range.y;
    if (us >= ue) return;

    // ------------------------------------------------- copies, units ahead
    // The warp's units of a piece are its begin + warp, + W, ..; pieces follow each other.
    Segment ps = find_segment(A, lay, us, kAtRows, kAtUnit);
    int pend = min(ps.u0 + ps.units, ue), pu = us + warp;
    int pages_l = -1, next = 0;                 // pages of the next 32 of the warp's units, one to a lane
    auto fetch_pages = [&]() {
        const int u = pu + lane * W;
        if (u < pend)
            pages_l = __ldg(A.b.table + static_cast<size_t>(ps.b) * A.b.max_pages + ((u - ps.u0) * kAtUnit >> A.c.lg));
        next = 0;
    };
    auto settle = [&]() {                       // pu: the next unit to order (or none: pu >= pend)
        if (pu >= pend) {
            if (pend >= ue) return;
            do {
                const int begin = pend;
                ps = find_segment(A, lay, begin, kAtRows, kAtUnit);
                pend = min(ps.u0 + ps.units, ue);
                pu = begin + warp;
            } while (pu >= pend && pend < ue);
            fetch_pages();
        } else if (next == 32) {
            fetch_pages();
        }
    };
    int issued = 0;
    auto order = [&](int slot) {
        if (pu >= pend) return;
        const uint32_t bar = bars + 8 * slot;
        const int page = __shfl_sync(0xffffffffu, pages_l, next);
        const bool there = page >= 0 && page < A.c.pages;
        if (lane == 0) {
            ok_s[slot] = there;
            if (there) {
                const int y = (pu - ps.u0) * kAtUnit & (A.c.page - 1);
                const int z = page * A.c.Hkv + ps.h;
                mbar_arrive_expect_tx(bar, C::kSlot + (CT == T_I8 ? 2 * kAtUnit * 4 : 0));
                const uint32_t dst = ring_a + slot * C::kSlot;
#pragma unroll
                for (int x = 0; x < C::kBoxes; ++x) {
                    tma_load_3d(dst + x * kAtUnit * C::kBox, &A.kmap, x * C::kBox / C::kEb, y, z, bar);
                    tma_load_3d(dst + C::kHalf + x * kAtUnit * C::kBox, &A.vmap, x * C::kBox / C::kEb, y, z, bar);
                }
                if constexpr (CT == T_I8) {
                    const size_t at = static_cast<size_t>(z) * A.c.page + y;
                    bulk_copy(smem_u32(scale_s + slot * 2 * kAtUnit), A.c.ks + at, kAtUnit * 4, bar);
                    bulk_copy(smem_u32(scale_s + slot * 2 * kAtUnit + kAtUnit), A.c.vs + at, kAtUnit * 4, bar);
                }
            } else {
                mbar_arrive(bar);
            }
        }
        __syncwarp();
        ++issued;
        ++next;
        pu += W;
        settle();
    };

    // ------------------------------------------------------------ segments
    int slot = 0, seen = 0;
    uint32_t phase = 0;
    bool dead = false;
    uint32_t qa[D / 16][4];
    unsigned long long see[2];
    auto load_rows = [&](const Segment& sg, int rows) {       // this lane's rows g and g + 8: queries, masks
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = g + 8 * e;
            const bool have = r < rows;
            const int rr = sg.tile * kAtRows + (have ? r : 0);
            const int tok = rr / A.G, t = sg.f.q0 + tok;
            see[e] = A.mask != nullptr ? __ldg(A.mask + t) : (2ull << tok) - 1ull;
            const uint16_t* q = static_cast<const uint16_t*>(A.q) + (static_cast<size_t>(t) * A.Hq + sg.h * A.G + (rr - tok * A.G)) * D;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                uint2 v = make_uint2(0u, 0u);
                if (have) {
                    if constexpr (CT == T_I8) { // a lane's K values of a step are four codes in a row
                        v = __ldg(reinterpret_cast<const uint2*>(q + 16 * j + 4 * c));
                    } else {
                        v.x = __ldg(reinterpret_cast<const unsigned*>(q + 16 * j + 2 * c));
                        v.y = __ldg(reinterpret_cast<const unsigned*>(q + 16 * j + 8 + 2 * c));
                    }
                }
                qa[j][e] = v.x;
                qa[j][2 + e] = v.y;
            }
        }
    };
    auto rows_of = [&](const Segment& sg) { return min(kAtRows, sg.f.n * A.G - sg.tile * kAtRows); };
    Segment sg = ps;
    fetch_pages();
    load_rows(sg, rows_of(sg));
    settle();
#pragma unroll 1
    for (int k = 0; k < C::kSlots; ++k) order(k);
#pragma unroll 1
    for (int begin = us; begin < ue;) {
        const int end = min(sg.u0 + sg.units, ue), rows = rows_of(sg);
        float o[D / 8][4];
#pragma unroll
        for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
        float m[2] = {neg_inf(), neg_inf()}, l[2] = {0.0f, 0.0f};

#pragma unroll 1
        for (int u = begin + warp; u < end; u += W) {
            if (!dead) {
                const bool ok = mbar_wait_bounded(bars + 8 * slot, phase, kAtWaitNs);
                if (!__all_sync(0xffffffffu, ok)) {
                    dead = true;
                    if (lane == 0 && A.err != nullptr) atomicExch(A.err, kErrWaitTimeout);
                }
            }
            if (dead) continue;
            ++seen;
            uint8_t* ks = ring + slot * C::kSlot;
            uint8_t* vs = ks + C::kHalf;
            const uint32_t ka = ring_a + slot * C::kSlot, va = ka + C::kHalf;
            const int t0 = (u - sg.u0) * kAtUnit;
            if (ok_s[slot] != 0) {
                // scores: tokens 2c, 2c + 1, 8 + 2c, 9 + 2c of rows g, g + 8
                float s[2][4] = {};
                if constexpr (CT == T_I8) {
#pragma unroll
                    for (int j = 0; j < D / 16; ++j)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t w = *reinterpret_cast<const uint32_t*>(ks + place_of<D, CT>(g + 8 * h, 16 * j + 4 * c));
                            uint32_t b0, b1;
                            codes16<QT>(w, b0, b1);
                            mma16<QT>(s[h], qa[j], b0, b1);
                        }
                } else {
                    // four 8 x 8 matrices: tokens 0-7 and 8-15, each the two halves of 16 columns
                    const int t = (lane & 7) + ((lane >> 4) << 3), x = (lane >> 3 & 1) * 16;
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        uint32_t b[4];
                        ldsm_x4(ka + place_of<D, CT>(t, 32 * j + x), b);
                        mma16<QT>(s[0], qa[j], b[0], b[1]);
                        mma16<QT>(s[1], qa[j], b[2], b[3]);
                    }
                }
                float vsc[4];
                if constexpr (CT == T_I8) {
                    const float* sc = scale_s + slot * 2 * kAtUnit;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float2 kk = *reinterpret_cast<const float2*>(sc + 8 * h + 2 * c);
                        const float2 vv = *reinterpret_cast<const float2*>(sc + kAtUnit + 8 * h + 2 * c);
                        s[h][0] *= kk.x * A.scale; s[h][2] *= kk.x * A.scale;
                        s[h][1] *= kk.y * A.scale; s[h][3] *= kk.y * A.scale;
                        vsc[2 * h] = vv.x;
                        vsc[2 * h + 1] = vv.y;
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int k = 0; k < 4; ++k) s[h][k] *= A.scale;
                }
                // drafts: a row sees those of its mask; places behind the last do not count
                const bool drafts = t0 + kAtUnit > sg.f.ctx;
                unsigned hidden = 0;
                if (drafts) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int t = t0 + 8 * h + 2 * c + (k & 1), j = t - sg.f.ctx;
                            if (j >= 0 && (t >= sg.f.len || ((see[k >> 1] >> j) & 1ull) == 0ull)) {
                                s[h][k] = neg_inf();
                                hidden |= 1u << (4 * h + k);
                            }
                        }
                }
                uint32_t pa[kParts][4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float top = fmaxf(fmaxf(s[0][2 * e], s[0][2 * e + 1]), fmaxf(s[1][2 * e], s[1][2 * e + 1]));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    if (__any_sync(0xffffffffu, top > m[e])) {
                        const float was = m[e];
                        m[e] = fmaxf(was, top);
                        const float f = was == neg_inf() ? 0.0f : exp2_fast(was - m[e]);
                        l[e] *= f;
#pragma unroll
                        for (int j = 0; j < D / 8; ++j) {
                            o[j][2 * e] *= f;
                            o[j][2 * e + 1] *= f;
                        }
                    }
                    const float base = (m[e] == neg_inf() ? 0.0f : m[e]) - kLift;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int k = 2 * e; k < 2 * e + 2; ++k) {
                            const float p = exp2_fast(s[h][k] - base);
                            l[e] += p;
                            if constexpr (CT == T_I8) s[h][k] = (hidden >> (4 * h + k)) & 1u ? 0.0f : p * vsc[2 * h + (k & 1)];
                            else s[h][k] = p;
                        }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = s[h][2 * e], y = s[h][2 * e + 1];
#pragma unroll
                        for (int k = 0; k < kParts; ++k) pa[k][2 * h + e] = part16<PT, CT == T_I8>(x, y, k + 1 == kParts);
                    }
                if constexpr (CT == T_I8 && kParts > 1) {
                    if (__any_sync(0xffffffffu, vast(vsc[0]) || vast(vsc[1]) || vast(vsc[2]) || vast(vsc[3])))
#pragma unroll
                        for (int k = 1; k < kParts; ++k)
#pragma unroll
                            for (int w = 0; w < 4; ++w) pa[k][w] = only_first(pa[k][w], vast(vsc[w & 2]), vast(vsc[(w & 2) + 1]));
                }
                // The tensor cores cut a sum's low bits at every step: for an output of more bits the units are added here.
                // (16 bits: 1024 steps are 1.0e-4 off if all values are positive, 0.4 half steps of fp16; added here, 64 streams of
                // two parts and D 64, 128, 256 take 78, 104, 160 us instead of 74, 103, 129.)
                auto pv = [&](float (&acc)[4], uint32_t b0, uint32_t b1) {
                    if constexpr (kAdd) {
                        float d[4] = {};
#pragma unroll
                        for (int k = kParts - 1; k >= 0; --k) mma16<PT>(d, pa[k], b0, b1);
#pragma unroll
                        for (int k = 0; k < 4; ++k) acc[k] += d[k];
                    } else {
#pragma unroll
                        for (int k = kParts - 1; k >= 0; --k) mma16<PT>(acc, pa[k], b0, b1);
                    }
                };
                if constexpr (CT == T_I8) {
                    // four tokens' words of four columns, transposed: columns 4 (g + 8 jj) + i of tokens 2c, 2c + 1, 8 + 2c, 9 + 2c
#pragma unroll
                    for (int jj = 0; jj < D / 32; ++jj) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            w[k] = *reinterpret_cast<const uint32_t*>(vs + place_of<D, CT>(2 * c + (k & 1) + 8 * (k >> 1), 4 * (g + 8 * jj)));
                        const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[2], w[3], 0x5140);
                        const uint32_t d = __byte_perm(w[0], w[1], 0x7362), e = __byte_perm(w[2], w[3], 0x7362);
                        const uint32_t col[4] = {__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632),
                                                 __byte_perm(d, e, 0x5410), __byte_perm(d, e, 0x7632)};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t b0, b1;
                            i8_to_bf16(col[i], b0, b1);
                            pv(o[4 * jj + i], b0, b1);
                        }
                    }
                } else {
                    bool plain = false;
                    if (drafts) {
                        // Places behind the last hold anything: zeros in their stead.  A draft's infinities and NaN would
                        // reach the rows that do not see it (0 times them): such a unit is summed without the tensor cores.
                        bool odd = false;
                        for (int k = lane; k < kAtUnit * D / 2; k += 32) {
                            const int t = k / (D / 2);
                            uint32_t* w = reinterpret_cast<uint32_t*>(vs + place_of<D, CT>(t, 4 * (k % (D / 2))));
                            const uint32_t top = CT == T_F16 ? 0x7c00u : 0x7f80u;
                            if (t0 + t >= sg.f.len) *w = 0u;
                            else if (t0 + t >= sg.f.ctx) odd |= (*w & top) == top || (*w >> 16 & top) == top;
                        }
                        plain = __any_sync(0xffffffffu, odd);
                        __syncwarp();
                    }
                    if (!plain) {
                        const int t = lane & 15, x = (lane >> 4) * 16;
#pragma unroll
                        for (int j = 0; j < D / 16; ++j) {
                            uint32_t b[4];
                            ldsm_x4_t(va + place_of<D, CT>(t, 32 * j + x), b);
                            pv(o[2 * j], b[0], b[1]);
                            pv(o[2 * j + 1], b[2], b[3]);
                        }
                    } else {
#pragma unroll 1
                        for (int t = 0; t < kAtUnit; ++t) {
                            const int from = (lane & 28) | ((t & 7) >> 1);
                            float p[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float p0 = __shfl_sync(0xffffffffu, t & 8 ? s[1][2 * e] : s[0][2 * e], from);
                                const float p1 = __shfl_sync(0xffffffffu, t & 8 ? s[1][2 * e + 1] : s[0][2 * e + 1], from);
                                p[e] = t & 1 ? p1 : p0;
                                const int j = t0 + t - sg.f.ctx;
                                if (j >= 0 && (t0 + t >= sg.f.len || ((see[e] >> j) & 1ull) == 0ull)) p[e] = -1.0f;
                            }
#pragma unroll
                            for (int j = 0; j < D / 8; ++j) {
                                const float2 v = unpair16<PT>(*reinterpret_cast<const uint32_t*>(vs + place_of<D, CT>(t, 2 * (8 * j + 2 * c))));
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (p[e] >= 0.0f) {
                                        o[j][2 * e] += p[e] * v.x;
                                        o[j][2 * e + 1] += p[e] * v.y;
                                    }
                            }
                        }
                    }
                    if (drafts) fence_proxy_async_smem();     // (zeros were written where the next copy lands)
                }
            }
            __syncwarp();
            order(slot);
            if (++slot == C::kSlots) {
                slot = 0;
                phase ^= 1u;
            }
        }

        // -------------------------------------------- the warps' results joined
        const Segment done = sg;
        if (end < ue) {                         // (the next queries are on their way meanwhile)
            sg = find_segment(A, lay, end, kAtRows, kAtUnit);
            load_rows(sg, rows_of(sg));
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            if (c == 0) {
                ml_s[(warp * 2) * kAtRows + g + 8 * e] = m[e];
                ml_s[(warp * 2 + 1) * kAtRows + g + 8 * e] = l[e];
            }
        }
        const bool lost = __syncthreads_or(dead) != 0;
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = g + 8 * e;
            float top = neg_inf(), sum = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) top = fmaxf(top, ml_s[w * 2 * kAtRows + r]);
            const float base = top == neg_inf() ? 0.0f : top;
#pragma unroll
            for (int w = 0; w < W; ++w) sum += ml_s[(w * 2 + 1) * kAtRows + r] * exp2_fast(ml_s[w * 2 * kAtRows + r] - base);
            f[e] = exp2_fast(m[e] - base);
            if (warp == 0 && c == 0) {
                fin_s[r] = top;
                fin_s[kAtRows + r] = sum;
            }
        }
        auto at = [&](int e, int j, int k) {                  // accumulator (row g + 8 e, tile j, column k) -> place in a joined row block
            const int d = CT == T_I8 ? 4 * (2 * c + k + 8 * (j >> 2)) + (j & 3) : 8 * j + 2 * c + k;
            return (g + 8 * e) * C::kPad + d;
        };
        // Behind the block's last unit the rings are free (every copy was waited for): a place for each warp.  Before, the
        // warps take turns on one or two.
        const bool idle = end == ue && !lost;
        float* area = idle ? reinterpret_cast<float*>(smem + C::oRing) : join_s;
        const int parts = idle ? W : C::kParts, turns = W / parts;
        float* mine = area + (warp % parts) * kAtRows * C::kPad;
#pragma unroll 1
        for (int turn = 0; turn < turns; ++turn) {
            if (warp / parts == turn) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (g + 8 * e < rows)
#pragma unroll
                        for (int j = 0; j < D / 8; ++j)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                float& v = mine[at(e, j, k)];
                                v = turn == 0 ? o[j][2 * e + k] * f[e] : v + o[j][2 * e + k] * f[e];
                            }
            }
            __syncthreads();
        }
        const bool whole = begin == done.u0 && end == done.u0 + done.units;
        float* part = A.part + (static_cast<size_t>(blockIdx.x) * 2 + (us < done.u0 ? 1 : 0)) * attn_part_floats(A.part_rows, D);
        if (!whole && tid < rows) {
            part[tid] = fin_s[tid];
            part[A.part_rows + tid] = fin_s[kAtRows + tid];
        }
        for (int k = tid; k < rows * (D / 4); k += C::kThreads) {
            const int r = k / (D / 4), d = k % (D / 4) * 4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (int w = 0; w < parts; ++w) {
                const float4 t = *reinterpret_cast<const float4*>(area + (w * kAtRows + r) * C::kPad + d);
                v.x += t.x; v.y += t.y; v.z += t.z; v.w += t.w;
            }
            if (!whole) {
                *reinterpret_cast<float4*>(part + 2 * A.part_rows + r * D + d) = v;
            } else {
                const float sum = fin_s[kAtRows + r], inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                const int rr = done.tile * kAtRows + r, tok = rr / A.G;
                const size_t y = (static_cast<size_t>(done.f.q0 + tok) * A.Hq + done.h * A.G + (rr - tok * A.G)) * D + d;
                const float w[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
                if (A.ytype == T_F32) *reinterpret_cast<float4*>(static_cast<float*>(A.y) + y) = make_float4(w[0], w[1], w[2], w[3]);
                else if (A.ytype == T_F16) *reinterpret_cast<uint2*>(static_cast<uint16_t*>(A.y) + y) = make_uint2(pair16<T_F16>(w[0], w[1]), pair16<T_F16>(w[2], w[3]));
                else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(A.y) + y) = make_uint2(pair16<T_BF16>(w[0], w[1]), pair16<T_BF16>(w[2], w[3]));
            }
        }
        __syncthreads();
        begin = end;
    }
    // after a timeout: this warp's copies in flight land before the block ends
    if (dead)
        for (int k = seen; k < issued; ++k)
            if (!mbar_wait_bounded(bars + 8 * (k % C::kSlots), static_cast<uint32_t>(k / C::kSlots) & 1u, kAtWaitNs)) break;
}

// Segments that several blocks share: their pieces' results, weighted by 2^(maximum - the largest) and added in a fixed
// order.  The grid has some blocks for each border between two blocks of the first launch.  A segment of p pieces has p - 1 borders inside, which
// deal its rows among them: a border's work is about the same whether a few segments are in many pieces or many in two.
// A row of few pieces is a warp's, of many the block's: eight warps, every eighth piece each, eight at a time.  Maximum, sum
// and values are loaded together, so a row costs one round of loads per 8 (or 64) pieces.
constexpr int kJoinWarps = 8, kJoinFew = 8;
template <int D>
struct JoinRow {
    static constexpr int kV = D / 32;
    float m, l, acc[kV];
};
// Pieces from, from + step, .. of a row.
template <int D>
__device__ __forceinline__ void join_pieces(JoinRow<D>& R, const float* first, const float* others, size_t pf, int part_rows,
                                            int row, int from, int step, int pieces, int lane)
{
    constexpr int kV = JoinRow<D>::kV, kBatch = 8;
    R.m = neg_inf();
    R.l = 0.0f;
#pragma unroll
    for (int v = 0; v < kV; ++v) R.acc[v] = 0.0f;
#pragma unroll 1
    for (int k0 = from; k0 < pieces; k0 += step * kBatch) {
        float pm[kBatch], pl[kBatch], pv[kBatch][kV];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
            pm[e] = neg_inf();
            pl[e] = 0.0f;
#pragma unroll
            for (int v = 0; v < kV; ++v) pv[e][v] = 0.0f;
            if (k0 + step * e < pieces) {
                const int k = k0 + step * e;
                const float* p = k == 0 ? first : others + 2 * k * pf;
                pm[e] = __ldcg(p + row);
                pl[e] = __ldcg(p + part_rows + row);
                const float* o = p + 2 * part_rows + row * D + kV * lane;
                if constexpr (kV == 2) {
                    const float2 v = __ldcg(reinterpret_cast<const float2*>(o));
                    pv[e][0] = v.x;
                    pv[e][1] = v.y;
                } else {
#pragma unroll
                    for (int q = 0; q < kV; q += 4) {
                        const float4 v = __ldcg(reinterpret_cast<const float4*>(o + q));
                        pv[e][q] = v.x; pv[e][q + 1] = v.y; pv[e][q + 2] = v.z; pv[e][q + 3] = v.w;
                    }
                }
            }
        }
        float top = R.m;
#pragma unroll
        for (int e = 0; e < kBatch; ++e) top = fmaxf(top, pm[e]);
        const float base = top == neg_inf() ? 0.0f : top, w = exp2_fast(R.m - base);
        R.m = top;
        R.l *= w;
#pragma unroll
        for (int v = 0; v < kV; ++v) R.acc[v] *= w;
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
            const float x = exp2_fast(pm[e] - base);          // (0 where nothing was seen; a sum that is NaN stays one)
            R.l += x * pl[e];
#pragma unroll
            for (int v = 0; v < kV; ++v) R.acc[v] += x * pv[e][v];
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) attn_join_kernel(const __grid_constant__ AttnArgs A, int tile_rows, int unit)
{
    constexpr int kV = D / 32;
    __shared__ __align__(16) float acc_s[kJoinWarps][D];
    __shared__ float m_s[kJoinWarps], l_s[kJoinWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_launch_dependents();
    Layout lay;
    if (A.b.B <= 32) {
        lay = lane_layout(A, tile_rows, unit, lane);
    } else {
        pdl_wait();
        lay.pre = A.head;
        lay.total = A.head[A.b.B];
        lay.share = max((lay.total + A.blocks - 1) / A.blocks, A.least);
        lay.mine = lay.n = lay.mine_b = lay.blocks = 0;
        lay.f = SeqFacts{0, 0, 0, 0};
    }
    // the border before block j: the one inside a segment whose pieces are those of blocks j0, j0 + 1, ..
    const int j = static_cast<int>(blockIdx.x) + 1;
    Segment sg = {};
    bool inside = false;
    int j0 = 0, pieces = 0;
    if (lay.share == 0) {
        const OwnPiece p = own_piece(lay, A, j, unit);
        inside = p.j > 0;
        if (inside) {
            sg = find_segment(A, lay, p.us, tile_rows, unit);
            j0 = j - p.j;
            pieces = p.n;
        }
    } else {
        const long long border = static_cast<long long>(j) * lay.share;
        if (border < lay.total) {
            sg = find_segment(A, lay, static_cast<int>(border), tile_rows, unit);
            inside = sg.u0 != border;
            j0 = sg.u0 / lay.share;
            pieces = (sg.u0 + sg.units - 1) / lay.share - j0 + 1;
        }
    }
    if (A.b.B <= 32) pdl_wait();                // (every thread: the launch ends behind the one before it)
    if (!inside) return;
    const int rows = min(tile_rows, sg.f.n * A.G - sg.tile * tile_rows);
    const size_t pf = attn_part_floats(A.part_rows, D);
    // (a block's first piece is in its first place, a segment that begins within the block in the second)
    const float* first = A.part + (static_cast<size_t>(j0) * 2 + (lay.share > 0 && j0 * lay.share < sg.u0 ? 1 : 0)) * pf;
    const float* others = A.part + static_cast<size_t>(j0) * 2 * pf;
    auto write = [&](const JoinRow<D>& R, int row) {
        const float inv = R.l == 0.0f ? 0.0f : 1.0f / R.l;
        const int rr = sg.tile * tile_rows + row, tok = rr / A.G;
        const size_t y = (static_cast<size_t>(sg.f.q0 + tok) * A.Hq + sg.h * A.G + (rr - tok * A.G)) * D + kV * lane;
#pragma unroll
        for (int v = 0; v < kV; ++v) store_typed(A.y, A.ytype, y + v, R.acc[v] * inv);
    };
    JoinRow<D> R;
    const int stride = pieces - 1, mine = j - 1 - j0;           // this border's rows: mine, mine + stride, ..
    if (pieces <= kJoinFew) {
#pragma unroll 1
        for (int row = mine + (static_cast<int>(blockIdx.y) * kJoinWarps + warp) * stride; row < rows;
             row += static_cast<int>(gridDim.y) * kJoinWarps * stride) {
            join_pieces<D>(R, first, others, pf, A.part_rows, row, 0, 1, pieces, lane);
            write(R, row);
        }
        return;
    }
#pragma unroll 1
    for (int row = mine + static_cast<int>(blockIdx.y) * stride; row < rows; row += static_cast<int>(gridDim.y) * stride) {
        join_pieces<D>(R, first, others, pf, A.part_rows, row, warp, kJoinWarps, pieces, lane);
        if (lane == 0) {
            m_s[warp] = R.m;
            l_s[warp] = R.l;
        }
#pragma unroll
        for (int v = 0; v < kV; ++v) acc_s[warp][kV * lane + v] = R.acc[v];
        __syncthreads();
        if (warp == 0) {
            float top = m_s[0];
#pragma unroll
            for (int w = 1; w < kJoinWarps; ++w) top = fmaxf(top, m_s[w]);
            const float base = top == neg_inf() ? 0.0f : top;
            R.l = 0.0f;
#pragma unroll
            for (int v = 0; v < kV; ++v) R.acc[v] = 0.0f;
#pragma unroll
            for (int w = 0; w < kJoinWarps; ++w) {
                const float x = exp2_fast(m_s[w] - base);
                R.l += x * l_s[w];
#pragma unroll
                for (int v = 0; v < kV; ++v) R.acc[v] += x * acc_s[w][kV * lane + v];
            }
            write(R, row);
        }
        __syncthreads();
    }
}

void dependent(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr)
{
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
}

constexpr int kExtra = 16;                      // (3 us at 185 ns a unit, measured on bf16 heads of 128)

template <int D, int CT, int QT, int kParts, bool kAdd>
cudaError_t launch(AttnArgs& a, int sms, cudaStream_t s)
{
    using C = At<D, CT>;
    auto kern = attn_tree_kernel<D, CT, QT, kParts, kAdd>;
    static SmemLimit limit;
    cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), limit, C::smem(kAtMaxSeq));
    if (e == cudaSuccess) e = encode_kv_map(&a.kmap, a, a.c.k, C::kBox, kAtUnit);
    if (e == cudaSuccess) e = encode_kv_map(&a.vmap, a, a.c.v, C::kBox, kAtUnit);
    if (e != cudaSuccess) return e;
    a.blocks = blocks_of(sms);
    a.extra = kExtra;
    a.least = C::kWarps;                        // a unit for each warp
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(a.blocks));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::smem(a.b.B);
    cfg.stream = s;
    dependent(cfg, attr);
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int D, int CT, int QT>
cudaError_t launch_w(AttnArgs& a, int sms, cudaStream_t s)
{
    if (a.ytype == T_F32) return launch<D, CT, QT, CT == T_F16 ? 2 : 3, true>(a, sms, s);
    if constexpr (CT == T_F16) {
        if (a.ytype == T_BF16) return launch<D, CT, QT, 1, false>(a, sms, s);
    } else {
        if (a.ytype == T_F16) return launch<D, CT, QT, 2, true>(a, sms, s);
    }
    // as many bits as the output has: the sums may stay on the tensor cores for 1024 steps of a warp, or 8192 where it is bf16
    const long long steps = 2 * (piece_units(a, blocks_of(sms), kAtUnit, kExtra) / At<D, CT>::kWarps + 1);
    return steps > (a.ytype == T_F16 ? 1024 : 8192) ? launch<D, CT, QT, 2, true>(a, sms, s) : launch<D, CT, QT, 2, false>(a, sms, s);
}

template <int D>
cudaError_t launch_d(AttnArgs& a, int qtype, int sms, cudaStream_t s)
{
    if (a.c.type == T_F16) return launch_w<D, T_F16, T_F16>(a, sms, s);
    if (a.c.type == T_BF16) return launch_w<D, T_BF16, T_BF16>(a, sms, s);
    return qtype == T_F16 ? launch_w<D, T_I8, T_F16>(a, sms, s) : launch_w<D, T_I8, T_BF16>(a, sms, s);
}

}  // namespace

cudaError_t encode_kv_map(CUtensorMap* map, const AttnArgs& a, const void* base, int box_bytes, int box_rows)
{
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static std::atomic<void*> cached{nullptr};
    void* fn = cached.load(std::memory_order_acquire);
    if (fn == nullptr) {
        cudaDriverEntryPointQueryResult got;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &got);
        if (e != cudaSuccess) return e;
        if (got != cudaDriverEntryPointSuccess || fn == nullptr) return cudaErrorNotSupported;
        cached.store(fn, std::memory_order_release);
    }
    const cuuint64_t eb = a.c.type == T_I8 ? 1 : 2;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.c.D), static_cast<cuuint64_t>(a.c.page),
                                static_cast<cuuint64_t>(a.c.pages) * a.c.Hkv};
    const cuuint64_t strides[2] = {a.c.D * eb, a.c.D * eb * a.c.page};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_bytes / eb), static_cast<cuuint32_t>(box_rows), 1};
    const cuuint32_t ones[3] = {1, 1, 1};
    const CUresult r = reinterpret_cast<Encode>(fn)(
        map, eb == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(base), dims, strides,
        box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t launch_attn_join(const AttnArgs& a, int rows, int unit, cudaStream_t s)
{
    if (a.blocks < 2) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(a.blocks - 1), a.part_rows <= 16 ? 1u : 4u);
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = s;
    dependent(cfg, attr);
    return cudaLaunchKernelEx(&cfg, a.c.D == 64 ? attn_join_kernel<64> : a.c.D == 128 ? attn_join_kernel<128> : attn_join_kernel<256>,
                              a, rows, unit);
}

cudaError_t launch_attn_tree(AttnArgs& a, int qtype, int sms, cudaStream_t s)
{
    return a.c.D == 64 ? launch_d<64>(a, qtype, sms, s) : a.c.D == 128 ? launch_d<128>(a, qtype, sms, s)
                                                                            : launch_d<256>(a, qtype, sms, s);
}

}  // namespace w4k
