// Penalties for repeated tokens, biases and grammar masks on rows of logits.
//
//   n: how often the row's sequence has generated v (the drafts on the row's
//   path among it); seen: n > 0 or v in the prompt
//   l = l > 0 ? l / rep : l rep    where seen
//   l = l - freq n - pres          where n > 0
//   l = l + bias (entries for the same v added in their order)
//   l = -inf                       where v is not allowed
// each step one fp32 operation, rounded to the logits' type at the end.
//
// One pass over the logits, no scratch in global memory: a block takes a slice of 8192
// entries of one row, reads the row's token history (a few KB to some hundred
// KB from L2, once per slice) and counts the slice's tokens in shared memory
// (integer atomics: the order does not matter), while the slice's logits are
// on their way into registers.
#include "attention.h"
#include "ptx.cuh"
#include "typed_io.cuh"

namespace w4k {
namespace {

// A counted entry: bit 0 in the prompt, bit 1 a bias, above them n.
constexpr int kPrompt = 1, kBias = 2, kOnce = 4;

struct LogitSmem {
    int count[kLgSlice];
    unsigned allowed[kLgSlice / 32];
    int bias_id[kLgMaxBias];
    float bias[kLgMaxBias];
    int nbias;
};

template <int T>
__global__ void __launch_bounds__(kLgThreads) logits_kernel(const LogitArgs A)
{
    extern __shared__ __align__(16) uint8_t raw[];
    LogitSmem& S = *reinterpret_cast<LogitSmem*>(raw);
    constexpr int kVec = T == T_F32 ? 4 : 8;                  // values of a 16-byte word
    constexpr int kIter = kLgSlice / (kVec * kLgThreads);
    const int tid = threadIdx.x, lane = tid & 31;
    pdl_launch_dependents();
    pdl_wait();
    const int row = static_cast<int>(blockIdx.x / static_cast<unsigned>(A.slices));
    const int lo = static_cast<int>(blockIdx.x - static_cast<unsigned>(row) * A.slices) * kLgSlice;
    const int n = min(kLgSlice, A.V - lo);
    int seq = row, first = row, last = row + 1;
    if (A.row_start != nullptr) {
        seq = row_sequence(A.row_start, A.S, row, lane);
        if (seq < A.S) {
            first = __ldg(A.row_start + seq);
            last = min(__ldg(A.row_start + seq + 1), A.R);
        }
    }
    if (seq >= A.S || row < first || first < 0) return;       // behind the last sequence

    // the slice's logits, on their way while the history is counted
    const size_t xat = static_cast<size_t>(row) * A.ld + lo;
    uint4 word[kIter];
    if (A.vec) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(A.x) + xat * elem_bytes(T));
#pragma unroll
        for (int k = 0; k < kIter; ++k) {
            const int w = k * kLgThreads + tid;
            word[k] = (w + 1) * kVec <= n ? p[w] : make_uint4(0u, 0u, 0u, 0u);
        }
    }
    const bool counted = A.ids != nullptr || A.drafts != nullptr || A.bias_ids != nullptr;
    for (int k = counted ? tid : kLgSlice; k < kLgSlice / 4; k += kLgThreads) reinterpret_cast<int4*>(S.count)[k] = make_int4(0, 0, 0, 0);
    if (A.allowed != nullptr) {
        const unsigned* bits = A.allowed + static_cast<size_t>(row) * ((A.V + 31) / 32) + lo / 32;
        for (int k = tid; k < (n + 31) / 32; k += kLgThreads) S.allowed[k] = __ldg(bits + k);
    }
    __syncthreads();
    auto count = [&](int id, int add) {
        const unsigned at = static_cast<unsigned>(id) - static_cast<unsigned>(lo);
        if (at < static_cast<unsigned>(n)) {
            if (add == kOnce) atomicAdd(&S.count[at], kOnce);
            else atomicOr(&S.count[at], add);
        }
    };
    if (A.ids != nullptr) {
        const int* ids = A.ids + static_cast<size_t>(seq) * A.cap;
        const int len = min(max(__ldg(A.length + seq), 0), A.cap);
        const int asked = A.prompt != nullptr ? __ldg(A.prompt + seq) : 0;
        if ((A.cap & 3) == 0 && (reinterpret_cast<uintptr_t>(A.ids) & 15u) == 0) {
#pragma unroll 4
            for (int k = tid; k < (len + 3) / 4; k += kLgThreads) {
                const int4 v = __ldg(reinterpret_cast<const int4*>(ids) + k);
                const int i = 4 * k;
                count(v.x, i < asked ? kPrompt : kOnce);
                if (i + 1 < len) count(v.y, i + 1 < asked ? kPrompt : kOnce);
                if (i + 2 < len) count(v.z, i + 2 < asked ? kPrompt : kOnce);
                if (i + 3 < len) count(v.w, i + 3 < asked ? kPrompt : kOnce);
            }
        } else {
            for (int k = tid; k < len; k += kLgThreads) count(__ldg(ids + k), k < asked ? kPrompt : kOnce);
        }
    }
    if (A.drafts != nullptr) {
        const int own = row - first;
        const unsigned long long m = A.mask != nullptr ? __ldg(A.mask + row) : 0ull;
        for (int j = tid; j < last - first; j += kLgThreads)
            if (A.mask != nullptr ? j < 64 && ((m >> j) & 1ull) != 0ull : j <= own) count(__ldg(A.drafts + first + j), kOnce);
    }
    if (A.bias_ids != nullptr && tid < 32) {
        // the slice's entries, in their order
        int at = 0;
        for (int k = 0; k < A.nb; k += 32) {
            int id = -1;
            float v = 0.0f;
            if (k + lane < A.nb) {
                id = __ldg(A.bias_ids + static_cast<size_t>(seq) * A.nb + k + lane);
                v = __ldg(A.bias + static_cast<size_t>(seq) * A.nb + k + lane);
            }
            const unsigned rel = static_cast<unsigned>(id) - static_cast<unsigned>(lo);
            const bool in = rel < static_cast<unsigned>(n);
            const unsigned who = __ballot_sync(0xffffffffu, in);
            if (in) {
                const int o = at + __popc(who & ((1u << lane) - 1u));
                S.bias_id[o] = static_cast<int>(rel);
                S.bias[o] = v;
                atomicOr(&S.count[rel], kBias);
            }
            at += __popc(who);
        }
        if (lane == 0) S.nbias = at;
    }
    __syncthreads();
    const float rep = A.rep != nullptr ? __ldg(A.rep + seq) : 1.0f;
    const float freq = A.freq != nullptr ? __ldg(A.freq + seq) : 0.0f;
    const float pres = A.pres != nullptr ? __ldg(A.pres + seq) : 0.0f;
    auto adjusted = [&](float v, int c, int at) {
        if (c != 0) {
            const int made = c >> 2;
            if (made > 0 || (c & kPrompt)) v = v > 0.0f ? __fdiv_rn(v, rep) : __fmul_rn(v, rep);
            if (made > 0) v = __fsub_rn(__fsub_rn(v, __fmul_rn(freq, static_cast<float>(made))), pres);
            if (c & kBias) {
                float add = 0.0f;
                for (int k = 0; k < S.nbias; ++k)
                    if (S.bias_id[k] == at) add = __fadd_rn(add, S.bias[k]);
                v = __fadd_rn(v, add);
            }
        }
        if (A.allowed != nullptr && ((S.allowed[at >> 5] >> (at & 31)) & 1u) == 0u) v = __int_as_float(0xff800000);
        return v;
    };
    const size_t yat = static_cast<size_t>(row) * A.ldy + lo;
    auto one_by_one = [&](int from) {
        for (int at = from; at < n; at += kLgThreads) {
            float v;
            if constexpr (T == T_F32) v = static_cast<const float*>(A.x)[xat + at];
            else if constexpr (T == T_F16) v = __half2float(static_cast<const __half*>(A.x)[xat + at]);
            else v = __bfloat162float(static_cast<const __nv_bfloat16*>(A.x)[xat + at]);
            store_typed(A.y, T, yat + at, adjusted(v, counted ? S.count[at] : 0, at));
        }
    };
    if (A.vec) {
        uint4* out = reinterpret_cast<uint4*>(static_cast<uint8_t*>(A.y) + yat * elem_bytes(T));
#pragma unroll
        for (int k = 0; k < kIter; ++k) {
            const int w = k * kLgThreads + tid, at = w * kVec;
            if (at + kVec > n) continue;
            int c[kVec] = {};
            if (counted) {
#pragma unroll
                for (int j = 0; j < kVec; j += 4) {
                    const int4 q = *reinterpret_cast<const int4*>(&S.count[at + j]);
                    c[j] = q.x; c[j + 1] = q.y; c[j + 2] = q.z; c[j + 3] = q.w;
                }
            }
            float v[kVec];
            const uint32_t r[4] = {word[k].x, word[k].y, word[k].z, word[k].w};
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                if constexpr (T == T_F32) v[j] = __uint_as_float(r[j]);
                else if constexpr (T == T_F16) v[j] = __half2float(__ushort_as_half(static_cast<unsigned short>(r[j / 2] >> (16 * (j & 1)))));
                else v[j] = __uint_as_float((j & 1) ? r[j / 2] & 0xffff0000u : r[j / 2] << 16);
                v[j] = adjusted(v[j], c[j], at + j);
            }
            uint4 o;
            if constexpr (T == T_F32) {
                o = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
            } else {
                uint32_t h[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (T == T_F16) {
                        const __half2 p = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
                        h[j] = *reinterpret_cast<const uint32_t*>(&p);
                    } else {
                        const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                        h[j] = *reinterpret_cast<const uint32_t*>(&p);
                    }
                }
                o = make_uint4(h[0], h[1], h[2], h[3]);
            }
            out[w] = o;
        }
        one_by_one(n / kVec * kVec + tid);                    // the row's end
        return;
    }
    one_by_one(tid);
}

template <int T>
cudaError_t launch(const LogitArgs& a, bool pdl, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.R) * static_cast<unsigned>(a.slices));
    cfg.blockDim = dim3(kLgThreads);
    cfg.dynamicSmemBytes = sizeof(LogitSmem);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    if (pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, logits_kernel<T>, a);
}

}  // namespace

static_assert(sizeof(LogitSmem) <= 48 * 1024, "no attribute is needed");

cudaError_t launch_logits(const LogitArgs& a, int type, bool pdl, cudaStream_t s)
{
    return type == T_F32 ? launch<T_F32>(a, pdl, s) : type == T_F16 ? launch<T_F16>(a, pdl, s) : launch<T_BF16>(a, pdl, s);
}

}  // namespace w4k
