// xq8_gemm.hip -- entry points of the product of rows in 8 bits (kernels:
// xq8_gemm.hpp).
#include "xsymv_host.hpp"
#include "xq8_gemm.hpp"
#include "xq8_host.hpp"

namespace xsymv {
namespace {

template <class T, int MT, int NT, int WK>
int stream_launch(const Q8GemmArgs<T>& g, hipStream_t stream)
{
    const long long blocks = (((long long)g.m + 16 * MT - 1) / (16 * MT)) *
                             (((long long)g.n + 16 * NT - 1) / (16 * NT));
    return q8_launch(&q8_gemm_stream<T, MT, NT, WK>, (unsigned)blocks, 64 * WK, stream, g);
}

template <class T, int BM, int BN, int WM, int WN, int S, int HOW>
int tile_launch(const Q8GemmArgs<T>& g, hipStream_t stream)
{
    const long long tiles = (((long long)g.m + BM - 1) / BM) * (((long long)g.n + BN - 1) / BN);
    return q8_launch(&q8_gemm_tile<T, BM, BN, WM, WN, S, HOW>, (unsigned)tiles, 64 * WM * WN, stream,
                     g);
}

// Rows at multiples of 16 bytes, and a tile's within 32-bit offsets.
inline bool rows_aligned(const signed char* p, int ld)
{
    return reinterpret_cast<size_t>(p) % 16 == 0 && ld % 16 == 0 && ld <= 1 << 23;
}

template <class T>
int gemm_run(int m, int n, int k, const signed char* a, int lda, const float* sa,
             const signed char* w, int ldw, const float* sw, const float* bias, T* c, int ldc,
             hipStream_t stream)
{
    if (m < 0) return -1;
    if (n < 0) return -2;
    if (k < 0 || k > Q8_MAX_K) return -3;
    const bool some = m > 0 && n > 0;
    if (some && k > 0 && a == nullptr) return -4;
    if (lda < std::max(1, k)) return -5;
    if (some && sa == nullptr) return -6;
    if (some && k > 0 && w == nullptr) return -7;
    if (ldw < std::max(1, k)) return -8;
    if (some && sw == nullptr) return -9;
    if (some && c == nullptr) return -11;
    if (ldc < std::max(1, n)) return -12;
    if (!some) return 0;
    const Q8GemmArgs<T> g{a, w, sa, sw, bias, c, lda, ldw, ldc, m, n, k, nullptr, 1, 1 << 30};
    if (m <= 16) return stream_launch<T, 1, 1, 4>(g, stream);
    if (m <= 32) return stream_launch<T, 2, 1, 4>(g, stream);
    if (m <= 64) return stream_launch<T, 4, 2, 4>(g, stream);
    if (rows_aligned(a, lda) && rows_aligned(w, ldw))
        return tile_launch<T, 256, 256, 2, 4, 2, Q8_LINES>(g, stream);
    return tile_launch<T, 256, 128, 4, 2, 2, Q8_REGS>(g, stream);
}

}  // namespace
}  // namespace xsymv

#define XSYMV_Q8_GEMM(L, CT, T)                                                                   \
    extern "C" int xsymv_q8gemm_##L(int m, int n, int k, const signed char* a, int lda,           \
                                    const float* sa, const signed char* w, int ldw,               \
                                    const float* sw, const float* bias, CT* c, int ldc,           \
                                    void* stream)                                                 \
    {                                                                                             \
        return xsymv::q8_guard([&] {                                                              \
            return xsymv::gemm_run<T>(m, n, k, a, lda, sa, w, ldw, sw, bias,                      \
                                      reinterpret_cast<T*>(c), ldc, (hipStream_t)stream);         \
        });                                                                                       \
    }

XSYMV_Q8_GEMM(s, float, float)
XSYMV_Q8_GEMM(h, xhalf, xsymv::q8half)
XSYMV_Q8_GEMM(b, xbfloat16, xsymv::q8bf16)
