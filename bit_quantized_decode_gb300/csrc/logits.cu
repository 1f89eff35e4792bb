// Penalties for repeated tokens, biases and grammar masks on rows of logits.
//
//   n: how often the row's sequence has generated v (the drafts on the row's
//   path among it); seen: n > 0 or v in the prompt
//   l = l > 0 ? l / rep : l rep    where seen
//   l = l - freq n - pres          where n > 0
//   l = l + the sum of v's biases (added up from 0 in their order)
//   l = -inf                       where v is not allowed
// each step one fp32 operation, rounded to the logits' type at the end.
//
// Two launches for two kinds of work.  The first copies the rows under the
// grammar's mask: pure streaming, nothing depends on the history (it is left
// out where the logits stay in place and no mask is given).  The second changes the few
// entries that the history, the drafts and the biases name: blocks of a row
// count its tokens, each those of its share of the hash values, in a hash table in shared memory while the first launch
// streams, wait for it, and rewrite each named entry once.  (One kernel that
// counts in dense slices had a block wait for its history in every slice: 200
// rows of 262144 with 1500 tokens took 100 us, 63 of them the bytes.)
// Integer counts: their order does not matter.
// 200 rows of 262144 fp32 logits under a grammar, 1500 tokens each: 87 us, the copy 62 of them (6.8 TB/s); rows of an odd width
// as fast.  One row of 152064 with 4096 tokens and 40 biases: 6.4 us.
#include "attention.h"
#include "ptx.cuh"
#include "typed_io.cuh"

namespace w4k {
namespace {

// A named entry: bit 0 in the prompt, bit 1 a bias, above them n.
constexpr int kPrompt = 1, kBias = 2, kOnce = 4;

// One value (a 16-bit type as its bits).
template <int T>
struct Cell {
    using type = uint16_t;
    static __device__ __forceinline__ float get(uint16_t v)
    {
        if constexpr (T == T_F16) return __half2float(__ushort_as_half(v));
        else return __uint_as_float(static_cast<uint32_t>(v) << 16);
    }
    static __device__ __forceinline__ uint16_t put(float f)
    {
        if constexpr (T == T_F16) return __half_as_ushort(__float2half_rn(f));
        else return __bfloat16_as_ushort(__float2bfloat16_rn(f));
    }
};
template <>
struct Cell<T_F32> {
    using type = float;
    static __device__ __forceinline__ float get(float v) { return v; }
    static __device__ __forceinline__ float put(float f) { return f; }
};

// Rows of the sequences; those behind are left alone.
__device__ __forceinline__ int live_rows(const LogitArgs& A)
{
    return A.row_start != nullptr ? min(__ldg(A.row_start + A.S), A.R) : min(A.S, A.R);
}

// ------------------------------------------------ rows copied under the mask
constexpr int kCopyVecs = 8;                    // 16-byte words of a thread
template <int T>
__global__ void __launch_bounds__(kLgThreads) logits_copy_kernel(const LogitArgs A)
{
    using V = typename Cell<T>::type;
    constexpr int kVec = 16 / sizeof(V), kBlock = kCopyVecs * kVec * kLgThreads;
    const V minus = Cell<T>::put(__int_as_float(0xff800000));
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_launch_dependents();                    // (behind the wait: the second launch reads its inputs early)
    const int row = static_cast<int>(blockIdx.x / static_cast<unsigned>(A.slices));
    const int slice = static_cast<int>(blockIdx.x - static_cast<unsigned>(row) * A.slices);
    const V* x = static_cast<const V*>(A.x) + static_cast<size_t>(row) * A.ld;
    V* y = static_cast<V*>(A.y) + static_cast<size_t>(row) * A.ldy;
    const unsigned* bits = A.allowed != nullptr ? A.allowed + static_cast<size_t>(row) * ((A.V + 31) / 32) : nullptr;
    auto one_by_one = [&](int from, int to) {
        for (int k = from; k < to; k += kLgThreads) y[k] = bits == nullptr || (__ldg(bits + (k >> 5)) >> (k & 31) & 1u) ? x[k] : minus;
    };
    if (!A.vec) {                               // x and y lie apart by no whole number of 16-byte words
        if (row < live_rows(A)) one_by_one(slice * kBlock + tid, min((slice + 1) * kBlock, A.V));
        return;
    }
    // 16-byte words begin `skew` values into the row (all rows of one width that is not a multiple of a word)
    const int skew = min(A.V, static_cast<int>((0 - reinterpret_cast<uintptr_t>(x)) % 16 / sizeof(V)));
    const int lo = skew + slice * kBlock, n = min(kBlock, A.V - lo);
    uint4 v[kCopyVecs];
    unsigned ok[kCopyVecs];
#pragma unroll
    for (int k = 0; k < kCopyVecs; ++k) {
        const int w = k * kLgThreads + tid;
        if ((w + 1) * kVec <= n) {
            v[k] = __ldcs(reinterpret_cast<const uint4*>(x + lo) + w);
            ok[k] = ~0u;
            if (bits != nullptr) {
                const int at = lo + w * kVec;
                ok[k] = __ldg(bits + (at >> 5)) >> (at & 31);
                if ((at & 31) + kVec > 32) ok[k] |= __ldg(bits + (at >> 5) + 1) << (32 - (at & 31));
            }
        }
    }
    if (row >= live_rows(A)) return;
#pragma unroll
    for (int k = 0; k < kCopyVecs; ++k) {
        const int w = k * kLgThreads + tid;
        if ((w + 1) * kVec <= n) {
            union {
                uint4 u;
                V e[kVec];
            } c;
            c.u = v[k];
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                if ((ok[k] >> j & 1u) == 0u) c.e[j] = minus;
            __stcs(reinterpret_cast<uint4*>(y + lo) + w, c.u);
        }
    }
    if (slice == 0) one_by_one(tid, skew);
    if (n > 0 && lo + n == A.V) one_by_one(lo + n / kVec * kVec + tid, A.V);  // the row's end
}

// --------------------------------------------------------- named entries
constexpr int kTouchThreads = 512, kTries = 64;
__device__ __forceinline__ unsigned mixed(int id) { return static_cast<unsigned>(id) * 2654435769u; }

template <int T>
__global__ void __launch_bounds__(kTouchThreads) logits_touch_kernel(const LogitArgs A, int lg_table, int lg_blocks, int behind_copy)
{
    using V = typename Cell<T>::type;
    extern __shared__ __align__(16) int table[];              // keys (-1: free), counts, then the biases
    const int size = 1 << lg_table;
    int* keys = table;
    int* counts = table + size;
    int* bias_id = counts + size;
    float* bias = reinterpret_cast<float*>(bias_id + A.nb);
    __shared__ int full;
    const int tid = threadIdx.x, lane = tid & 31, row = static_cast<int>(blockIdx.x >> lg_blocks);
    if (!behind_copy) pdl_wait();
    pdl_launch_dependents();
    int seq = row, first = row, last = row + 1;
    bool ours = row < live_rows(A);
    if (A.row_start != nullptr && ours) {
        seq = min(row_sequence(A.row_start, A.S, row, lane), A.S - 1);
        first = __ldg(A.row_start + seq);
        last = min(__ldg(A.row_start + seq + 1), A.R);
        ours = first >= 0 && row >= first && row < last;
    }
    if (!ours) {
        if (behind_copy) pdl_wait();            // (every block: the launch ends behind the first one)
        return;
    }
    const float rep = A.rep != nullptr ? __ldg(A.rep + seq) : 1.0f;
    const float freq = A.freq != nullptr ? __ldg(A.freq + seq) : 0.0f;
    const float pres = A.pres != nullptr ? __ldg(A.pres + seq) : 0.0f;
    int len = 0, asked = 0;
    const int* ids = A.ids + static_cast<size_t>(seq) * A.cap;
    if (A.ids != nullptr) {
        len = min(max(__ldg(A.length + seq), 0), A.cap);
        asked = A.prompt != nullptr ? __ldg(A.prompt + seq) : 0;
    }
    const bool quads = (A.cap & 3) == 0 && (reinterpret_cast<uintptr_t>(A.ids) & 15u) == 0;
    const V* x = static_cast<const V*>(A.x) + static_cast<size_t>(row) * A.ld;
    V* y = static_cast<V*>(A.y) + static_cast<size_t>(row) * A.ldy;
    const unsigned* bits = A.allowed != nullptr ? A.allowed + static_cast<size_t>(row) * ((A.V + 31) / 32) : nullptr;
    for (int k = tid; k < A.nb; k += kTouchThreads) {
        bias_id[k] = __ldg(A.bias_ids + static_cast<size_t>(seq) * A.nb + k);
        bias[k] = __ldg(A.bias + static_cast<size_t>(seq) * A.nb + k);
    }

    // This block's tokens: those whose hash ends in its number.  Where some token finds no place in the table, they are taken
    // in two halves by the next bit of the hash, and those in halves again: depth first, `prefix` the bits of the part at hand.
    // (The hash's lower bits are the id's times an odd number: 24 of them tell all ids apart.)
    const unsigned mine = blockIdx.x & ((1u << lg_blocks) - 1u);
    int depth = 0;
    unsigned prefix = 0;
    bool waited = !behind_copy;
    while (true) {
        for (int k = tid; k < size; k += kTouchThreads) {
            keys[k] = -1;
            counts[k] = 0;
        }
        if (tid == 0) full = 0;
        __syncthreads();
        const unsigned ending = mine | prefix << lg_blocks, ends = (1u << (lg_blocks + depth)) - 1u;
        auto add = [&](int id, int what) {
            const unsigned h = mixed(id);
            if (static_cast<unsigned>(id) >= static_cast<unsigned>(A.V) || (h & ends) != ending) return;
            unsigned at = h >> (32 - lg_table);
            for (int tries = 0; tries < kTries; ++tries, at = (at + 1) & (size - 1)) {
                int key = *reinterpret_cast<volatile int*>(&keys[at]);
                if (key == -1) {
                    key = atomicCAS(&keys[at], -1, id);
                    if (key == -1) key = id;
                }
                if (key == id) {
                    if (what == kOnce) atomicAdd(&counts[at], kOnce);
                    else atomicOr(&counts[at], what);
                    return;
                }
            }
            full = 1;
        };
        if (quads) {
            constexpr int kAhead = 4;           // loads in flight
#pragma unroll 1
            for (int i0 = 4 * tid; i0 < len; i0 += 4 * kTouchThreads * kAhead) {
                int4 v[kAhead];
#pragma unroll
                for (int e = 0; e < kAhead; ++e) {
                    const int i = i0 + 4 * kTouchThreads * e;
                    v[e] = i < len ? __ldg(reinterpret_cast<const int4*>(ids + i)) : make_int4(-1, -1, -1, -1);
                }
#pragma unroll
                for (int e = 0; e < kAhead; ++e) {
                    const int i = i0 + 4 * kTouchThreads * e;
                    if (i < len) add(v[e].x, i < asked ? kPrompt : kOnce);
                    if (i + 1 < len) add(v[e].y, i + 1 < asked ? kPrompt : kOnce);
                    if (i + 2 < len) add(v[e].z, i + 2 < asked ? kPrompt : kOnce);
                    if (i + 3 < len) add(v[e].w, i + 3 < asked ? kPrompt : kOnce);
                }
            }
        } else {
            for (int k = tid; k < len; k += kTouchThreads) add(__ldg(ids + k), k < asked ? kPrompt : kOnce);
        }
        if (A.drafts != nullptr) {
            const unsigned long long m = A.mask != nullptr ? __ldg(A.mask + row) : 0ull;
            for (int j = tid; j < last - first; j += kTouchThreads)
                if (A.mask != nullptr ? j < 64 && ((m >> j) & 1ull) != 0ull : j <= row - first) add(__ldg(A.drafts + first + j), kOnce);
        }
        for (int k = tid; k < A.nb; k += kTouchThreads) add(bias_id[k], kBias);
        __syncthreads();
        const bool again = *reinterpret_cast<volatile int*>(&full) != 0;
        __syncthreads();
        if (again) {
            ++depth;
            continue;
        }
        if (!waited) {
            pdl_wait();
            waited = true;
        }
        constexpr int kAhead = 4;               // entries' loads in flight
#pragma unroll 1
        for (int k0 = tid; k0 < size; k0 += kTouchThreads * kAhead) {
            int id[kAhead];
            V xv[kAhead];
#pragma unroll
            for (int e = 0; e < kAhead; ++e) {
                const int k = k0 + kTouchThreads * e;
                id[e] = k < size ? keys[k] : -1;
                if (id[e] >= 0) {
                    const unsigned ok = bits == nullptr ? 1u : __ldg(bits + (id[e] >> 5)) >> (id[e] & 31) & 1u;
                    xv[e] = x[id[e]];
                    if (ok == 0u) id[e] = -1;
                }
            }
#pragma unroll
            for (int e = 0; e < kAhead; ++e) {
                if (id[e] < 0) continue;
                const int c = counts[k0 + kTouchThreads * e], made = c >> 2;
                float v = Cell<T>::get(xv[e]);
                if (made > 0 || (c & kPrompt)) v = v > 0.0f ? __fdiv_rn(v, rep) : __fmul_rn(v, rep);
                if (made > 0) v = __fsub_rn(__fsub_rn(v, __fmul_rn(freq, static_cast<float>(made))), pres);
                if (c & kBias) {
                    float sum = 0.0f;
#pragma unroll 8
                    for (int j = 0; j < A.nb; ++j) sum = bias_id[j] == id[e] ? __fadd_rn(sum, bias[j]) : sum;
                    v = __fadd_rn(v, sum);
                }
                y[id[e]] = Cell<T>::put(v);
            }
        }
        while (depth > 0 && (prefix >> (depth - 1) & 1u) != 0u) {             // the second half is done: so is the part
            --depth;
            prefix &= ~(1u << depth);
        }
        if (depth == 0) break;
        prefix |= 1u << (depth - 1);
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

template <int T>
cudaError_t launch(LogitArgs& a, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    const bool copy = a.allowed != nullptr || a.x != a.y;
    if (copy) {
        constexpr int kBlock = kCopyVecs * (16 / elem_bytes(T)) * kLgThreads;
        a.slices = (a.V + kBlock - 1) / kBlock;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(a.R) * static_cast<unsigned>(a.slices));
        cfg.blockDim = dim3(kLgThreads);
        cfg.stream = s;
        dependent(cfg, attr);
        const cudaError_t e = cudaLaunchKernelEx(&cfg, logits_copy_kernel<T>, a);
        if (e != cudaSuccess) return e;
    }
    if (a.ids == nullptr && a.drafts == nullptr && a.bias_ids == nullptr) return cudaSuccess;
    // Blocks of a row: as many as keep a table's tokens to some 4096, or more while two blocks per SM are not there and a
    // block has more than 256.  A table twice as large as its share of the tokens, 512 to 16384 entries (128 KB).
    const long long most = static_cast<long long>(a.cap) + (a.drafts != nullptr ? 64 : 0) + a.nb;
    int lg_blocks = 0, lg = 9;
    while (lg_blocks < 8 && ((most >> lg_blocks) > 4096 || ((most >> lg_blocks) > 256 && (static_cast<long long>(a.R) << lg_blocks) < 152))) ++lg_blocks;
    while (lg < 14 && (1ll << lg) < 2 * (most >> lg_blocks)) ++lg;
    const size_t smem = 8 * (static_cast<size_t>(1) << lg) + 8 * static_cast<size_t>(a.nb);
    auto kern = logits_touch_kernel<T>;
    static SmemLimit limit;
    const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), limit, 8 * (1 << 14) + 8 * kLgMaxBias);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.R) << lg_blocks);
    cfg.blockDim = dim3(kTouchThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    dependent(cfg, attr);
    return cudaLaunchKernelEx(&cfg, kern, a, lg, lg_blocks, copy ? 1 : 0);
}

}  // namespace

cudaError_t launch_logits(LogitArgs& a, int type, cudaStream_t s)
{
    return type == T_F32 ? launch<T_F32>(a, s) : type == T_F16 ? launch<T_F16>(a, s) : launch<T_BF16>(a, s);
}

}  // namespace w4k
