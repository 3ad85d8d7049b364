// kv_cache.cu -- keys and values into the paged cache as codes, and back.
//
// Write: z = R x (RPBH rotation of a head's row), s = ||z||, codes = nearest centroids of
// sqrt(d) z / (s + eps), packed LSB-first; the same steps as the activation quantizer, on rows of
// one head, scattered by slot.  Read: x_hat = s / sqrt(d) R^T centroid[code].
//
// One warp a row: the gather through shared memory, the butterflies in registers and shuffles.  For few
// rows, where one launch's latency is the time: 8 tokens of 8 heads of 128 at 4 bits, write 3.3 us, read
// 2.5 us.  (Many 16-bit rows: kv_tc.cu.)
#include "k1_ops.cuh"
#include "kv_internal.h"
#include "kv_ops.cuh"
#include "kv_rows.cuh"

namespace oq {
namespace {

using namespace kvops;
using k1ops::fma_sat;

__device__ unsigned int g_kv_err;

constexpr int kWarps = 4;

// Row index -> (which of keys / values, token, head); token-major so that a token's heads, which
// lie together, are taken together.
struct Row {
    int w, head;
    long long tok;
};
__device__ __forceinline__ Row row_of(long long r, int heads) {
    Row o;
    o.head = (int)(r % heads);
    r /= heads;
    o.w = (int)(r & 1);
    o.tok = r >> 1;
    return o;
}

template <class E, int D>
__global__ void __launch_bounds__(32 * kWarps) kv_write_rows(const KvWriteParams p) {
    constexpr int N = D / 32;
    __shared__ float xs[kWarps][D];
    __shared__ __align__(16) uint8_t cs[kWarps][D];
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t ent[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        ent[i] = p.ent[lane * N + i];
    pdl_wait();
    const long long rows = 2ll * p.T * p.c.kv_heads;
    for (long long r = (long long)blockIdx.x * kWarps + warp; r < rows;
         r += (long long)gridDim.x * kWarps) {
        const Row o = row_of(r, p.c.kv_heads);
        const long long slot = p.slots[o.tok];
        if (!slot_ok(p.c, slot)) {
            if (slot != -1 && lane == 0)
                atomicOr(p.err, KV_ERR_SLOT);
            continue;
        }
        const E *x = static_cast<const E *>(pick(p.x, o.w)) + o.tok * pick(p.x_stride, o.w) + o.head * D;
#pragma unroll
        for (int i = 0; i < N; ++i)
            xs[warp][i * 32 + lane] = to_f32(x[i * 32 + lane]);
        __syncwarp();
        float z[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float v = xs[warp][ent[i] & 0x7fffu];
            z[i] = (ent[i] & 0x8000u) ? -v : v;
        }
        warp_wht<D>(z, p.h, lane);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i)
            sum += z[i] * z[i];
#pragma unroll
        for (int s = 16; s; s >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, s);
        const float norm = sqrtf(sum / (float)p.h);
        const float k = p.K / (norm + p.eps);
        uint32_t beside = 0;                             // bit i: a second look
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float a = fma_sat(z[i], k, 0.5f);
            const uint32_t q = __float_as_uint(__fadd_rd(a, 1.0f));
            const uint32_t word = p.tbl[((q - 0x3F800000u) >> p.F) * p.tbl_copies];
            const uint32_t at = word + q * (uint32_t)p.G;
            uint32_t code = at >> 24;
            if (distance_to_bound(at, p.G) < bound_width(p.G)) {
                if (z[i] == 0.f)
                    code = code_of_zero(p.c.bits);
                else
                    beside |= 1u << i;
            }
            cs[warp][lane * N + i] = (uint8_t)code;
        }
        beside = looks(norm) ? beside : 0u;
        __syncwarp();
        int left = kLooks;
#pragma unroll 1
        for (uint32_t any = __reduce_or_sync(0xffffffffu, beside); any; any &= any - 1) {
            const int i = __ffs(any) - 1;
#pragma unroll 1
            for (uint32_t lanes = __ballot_sync(0xffffffffu, (beside >> i) & 1u); lanes && left > 0;
                 lanes &= lanes - 1, --left) {
                const int at = (__ffs(lanes) - 1) * N + i;
                double sum = 0.0, squares = 0.0;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int pos = lane * N + j;
                    const double v = xs[warp][ent[j] & 0x7fffu];
                    squares += v * v;
                    if ((pos ^ at) < p.h)                // in one block
                        sum += ((ent[j] >> 15) ^ __popc(pos & at & (p.h - 1))) & 1u ? -v : v;
                }
                const uint32_t code = code_beside(cs[warp][at], sum, squares, norm, p.unit, p.bounds,
                                                  p.c.bits);
                __syncwarp();
                if (lane == 0)
                    cs[warp][at] = (uint8_t)code;
            }
        }
        __syncwarp();
        const long long at = cache_row(p.c, slot, o.head);
        if (lane == 0)
            pick(p.c.norms, o.w)[at] = norm;
        uint32_t *dst = reinterpret_cast<uint32_t *>(pick(p.c.codes, o.w) + at * p.c.row_bytes);
        for (int w = lane; w < p.c.row_bytes / 4; w += 32) {
            uint32_t v = 0;
            // codes that overlap bits [32 w, 32 w + 32)
            for (int c = 32 * w / p.c.bits; c * p.c.bits < 32 * w + 32; ++c) {
                const int sh = c * p.c.bits - 32 * w;
                const uint32_t code = cs[warp][c];
                v |= sh >= 0 ? code << sh : code >> -sh;
            }
            dst[w] = v;
        }
        __syncwarp();
    }
}

template <class E, int D>
__global__ void __launch_bounds__(32 * kWarps) kv_read_rows(const KvReadParams p) {
    constexpr int N = D / 32;
    __shared__ float xs[kWarps][D];
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t ent[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        ent[i] = p.ent[lane * N + i];
    pdl_wait();
    const long long rows = 2ll * p.T * p.c.kv_heads;
    for (long long r = (long long)blockIdx.x * kWarps + warp; r < rows;
         r += (long long)gridDim.x * kWarps) {
        const Row o = row_of(r, p.c.kv_heads);
        const long long slot = p.slots[o.tok];
        E *y = static_cast<E *>(pick(p.y, o.w)) + o.tok * pick(p.y_stride, o.w) + o.head * D;
        if (!slot_ok(p.c, slot)) {
            if (slot != -1 && lane == 0)
                atomicOr(p.err, KV_ERR_SLOT);
#pragma unroll
            for (int i = 0; i < N; ++i)
                y[i * 32 + lane] = from_f32<E>(0.f);
            continue;
        }
        const long long at = cache_row(p.c, slot, o.head);
        const uint8_t *row = pick(p.c.codes, o.w) + at * p.c.row_bytes;
        float z[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            z[i] = p.cent[code_at(row, lane * N + i, p.c.bits)];
        warp_wht<D>(z, p.h, lane);
        const float s = pick(p.c.norms, o.w)[at] * p.scale;
#pragma unroll
        for (int i = 0; i < N; ++i)
            xs[warp][ent[i] & 0x7fffu] = s * ((ent[i] & 0x8000u) ? -z[i] : z[i]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < N; ++i)
            y[i * 32 + lane] = from_f32<E>(xs[warp][i * 32 + lane]);
        __syncwarp();
    }
}

unsigned blocks_for(long long rows, int num_sms) {
    const long long want = (rows + kWarps - 1) / kWarps, most = 16ll * num_sms;
    return (unsigned)(want < most ? want : most);
}

template <class E>
cudaError_t write_rows(const KvWriteParams &p, cudaStream_t st, int num_sms) {
    const dim3 grid(blocks_for(2ll * p.T * p.c.kv_heads, num_sms)), block(32 * kWarps);
    if (p.c.d == 128)
        return launch_pdl(kv_write_rows<E, 128>, grid, block, 0, st, p);
    return launch_pdl(kv_write_rows<E, 256>, grid, block, 0, st, p);
}

template <class E>
cudaError_t read_rows(const KvReadParams &p, cudaStream_t st, int num_sms) {
    const dim3 grid(blocks_for(2ll * p.T * p.c.kv_heads, num_sms)), block(32 * kWarps);
    if (p.c.d == 128)
        return launch_pdl(kv_read_rows<E, 128>, grid, block, 0, st, p);
    return launch_pdl(kv_read_rows<E, 256>, grid, block, 0, st, p);
}

}  // namespace

namespace {

cudaError_t error_word(unsigned **out) {
    static PerDevice known;
    static void *word[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = known.once([&] { return cudaGetSymbolAddress(&word[dev], g_kv_err); });
    if (e == cudaSuccess)
        *out = static_cast<unsigned *>(word[dev]);
    return e;
}

// Rows (keys and values) from which the tensor cores' form is taken.  It and a warp a row, write (read),
// us: d = 128, 4 bits, 4096 rows 7.2 and 6.0 (4.4 and 3.7), 8192 rows 7.3 and 8.5 (4.4 and 5.1), 16384
// rows 8.0 and 13.2 (5.6 and 7.7); d = 256, 2 bits, 4096 rows 7.8 and 7.0 (5.7 and 4.5), 16384 rows 9.1
// and 17.2 (7.6 and 11.0).
constexpr long long kTensorRows = 8192;

}  // namespace

cudaError_t launch_kv_write(const KvWriteParams &params, int dtype, cudaStream_t st, int num_sms,
                            std::string *why) {
    *why = "oq_kv_write: launch";
    KvWriteParams p = params;
    const cudaError_t e = error_word(&p.err);
    if (e != cudaSuccess)
        return e;
    if (dtype == OQ_F32)
        return write_rows<float>(p, st, num_sms);
    if (2ll * p.T * p.c.kv_heads >= kTensorRows)
        return launch_kv_write_tc(p, p.r_img, p.tbl_words, dtype == OQ_BF16, st, num_sms);
    if (dtype == OQ_BF16)
        return write_rows<__nv_bfloat16>(p, st, num_sms);
    return write_rows<__half>(p, st, num_sms);
}

cudaError_t launch_kv_read(const KvReadParams &params, int dtype, cudaStream_t st, int num_sms,
                           std::string *why) {
    *why = "oq_kv_read: launch";
    KvReadParams p = params;
    const cudaError_t e = error_word(&p.err);
    if (e != cudaSuccess)
        return e;
    if (dtype == OQ_F32)
        return read_rows<float>(p, st, num_sms);
    if (2ll * p.T * p.c.kv_heads >= kTensorRows) {
        p.scale *= p.alpha_inv;
        return launch_kv_read_tc(p, p.r_img, dtype == OQ_BF16, st, num_sms);
    }
    if (dtype == OQ_BF16)
        return read_rows<__nv_bfloat16>(p, st, num_sms);
    return read_rows<__half>(p, st, num_sms);
}

cudaError_t read_and_clear_kv_error(unsigned *out, cudaStream_t st) {
    unsigned zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_kv_err, sizeof(unsigned), 0,
                                              cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess)
        e = cudaMemcpyToSymbolAsync(g_kv_err, &zero, sizeof(unsigned), 0,
                                    cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(st);
    return e;
}

}  // namespace oq
