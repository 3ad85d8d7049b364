// rope.cu -- rotary positions of queries and keys.
//
// Pair (a, b) of a head at position t becomes m (a cos - b sin, a sin + b cos) with the angle
// t * freq_i; the gradient goes back through the transpose, the same with -sin.  Bound by memory:
// each element is read and written once, 16 bytes at a time, and a block forms the cosines of its
// tokens once for all their heads.  Angles are taken in fp64 turns (t * freq / 2 pi minus its
// nearest integer), since an fp32 product at position 1e5 is already off by 1e-2 radians; the
// cosine itself is fp32: sincospif of the reduced turns in fp32, turned on by what that leaves of them
// (which costs nothing, and without it the turns' rounding is the largest error of fp32 rows).
// B200: 8192 tokens of 40 heads of 128, half of each turned in adjacent pairs, bf16: 28.2 us, 5.9 TB/s
// (0.91 of the measured copy rate); 4099 tokens of 48 heads in fp32: 31.9 us, 6.3 TB/s (0.96).
#include "kv_internal.h"
#include "kv_ops.cuh"

namespace oq {
namespace {

using namespace kvops;

constexpr int kThreads = 256;

// n / d for n < 2^23 and d < 2^17: with m = ceil(2^40 / d), n m / 2^40 passes n / d by less than 1 / d.
struct Divide {
    unsigned long long m;
    int d;
    explicit Divide(int by) : m(((1ull << 40) + by - 1) / by), d(by) {}
    __device__ __forceinline__ int operator()(int n) const { return (int)((n * m) >> 40); }
};

template <bool HALF> __host__ __device__ constexpr int ahead() { return HALF ? 2 : 4; }

// A block's work is a list of 16-byte vectors that turn (at HALF, each with its partner half a turned
// part away), then a list of those that are copied.  The cosines of a token lie in the order in
// which the vectors of a head take them, element by element, so that neighbouring lanes read
// neighbours.
template <class E, bool HALF>
__global__ void __launch_bounds__(kThreads, 5)
rope_kernel(const RopeParams p, const int tokens_a_block, const Divide by_turned,
            const Divide by_copied, const Divide by_heads) {
    extern __shared__ float2 cs[];                       // [tokens][e][vector]: (cos, sin)
    pdl_trigger();
    constexpr int V = Vec<E>::n, A = HALF ? V : V / 2;   // A angles a vector
    const int half = p.rot / 2;
    const int t0 = blockIdx.x * tokens_a_block;
    const int nt = min(tokens_a_block, p.T - t0);
    const int turned = by_turned.d, copied = by_copied.d, heads = by_heads.d;
    constexpr int kAhead = ahead<HALF>();                // vectors under way in a thread

    // Row r (a token's head) of the block's: its input and output.
    auto row = [&](int r, int t, const E *&x, E *&y) {
        int head = r - t * heads;
        const int w = head >= p.heads[0];
        head -= w ? p.heads[0] : 0;
        const long long tok = t0 + t;
        x = static_cast<const E *>(pick(p.x, w)) + tok * pick(p.x_stride, w) + head * p.d;
        y = static_cast<E *>(pick(p.y, w)) + tok * pick(p.y_stride, w) + head * p.d;
    };

    const int turns = nt * heads * turned;
    uint4 u[kAhead], v[HALF ? kAhead : 1];
    E *to[kAhead];
    int angle[kAhead];                                   // first of its angles
    auto load = [&](int k, int i) {
        if (i >= turns)
            return;
        const int r = by_turned(i), j = i - r * turned, t = by_heads(r);
        const E *x;
        row(r, t, x, to[k]);
        x += j * V;
        to[k] += j * V;
        angle[k] = t * half + j;
        u[k] = *reinterpret_cast<const uint4 *>(x);
        if (HALF)
            v[HALF ? k : 0] = *reinterpret_cast<const uint4 *>(x + half);
    };
    auto finish = [&](int k) {
        const float2 *a = cs + angle[k];
        float f[V];
        Vec<E>::unpack(u[k], f);
        if constexpr (HALF) {
            float g[V];
            Vec<E>::unpack(v[HALF ? k : 0], g);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float2 q = a[e * turned];
                const float x = f[e], y = g[e];
                f[e] = x * q.x - y * q.y;
                g[e] = x * q.y + y * q.x;
            }
            *reinterpret_cast<uint4 *>(to[k] + half) = Vec<E>::pack(g);
        } else {
#pragma unroll
            for (int e = 0; e < A; ++e) {
                const float2 q = a[e * turned];
                const float x = f[2 * e], y = f[2 * e + 1];
                f[2 * e] = x * q.x - y * q.y;
                f[2 * e + 1] = x * q.y + y * q.x;
            }
        }
        *reinterpret_cast<uint4 *>(to[k]) = Vec<E>::pack(f);
    };

    pdl_wait();
    // the first vectors are on their way while the angles are formed
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
        load(k, threadIdx.x + k * kThreads);
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int t = i / half, n = i - t * half;
        double turn = (double)p.pos[t0 + t] * p.turns[n];
        turn -= rint(turn);
        const float near = (float)turn, rest = 6.2831853f * (float)(turn - (double)near);
        float s, c;
        sincospif(2.0f * near, &s, &c);
        const float a = fmaf(-rest, s, c), b = fmaf(rest, c, s);
        cs[t * half + (n % A) * turned + n / A] =
            make_float2(p.amplitude * a, p.inverse ? -p.amplitude * b : p.amplitude * b);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < turns; i += kAhead * kThreads) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (i + k * kThreads < turns)
                finish(k);
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            load(k, i + (kAhead + k) * kThreads);
    }
    const int copies = p.d > p.rot ? nt * heads * copied : 0;
    for (int i = threadIdx.x; i < copies; i += 4 * kThreads) {
        uint4 c[4];
        E *out[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int n = i + k * kThreads;
            out[k] = nullptr;
            if (n >= copies)
                continue;
            const int r = by_copied(n), j = n - r * copied, t = by_heads(r);
            const E *x;
            E *y;
            row(r, t, x, y);
            if (x == y)
                continue;
            c[k] = *reinterpret_cast<const uint4 *>(x + p.rot + j * V);
            out[k] = y + p.rot + j * V;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (out[k] != nullptr)
                *reinterpret_cast<uint4 *>(out[k]) = c[k];
    }
}

template <class E>
cudaError_t run(const RopeParams &p, int layout, cudaStream_t st, int num_sms) {
    // Tokens a block: about one round of its threads' vectors, no more than one round of angles,
    // and few enough for two blocks an SM.  (8192 tokens of 40 heads, half of 128 elements turned:
    // 2, 3, 4, 8 tokens take 31.2, 28.6, 30.4, 34.6 us; 4099 of 48 in fp32: 1, 2, 4 take 31.9, 32.8,
    // 36.2 us.  48 registers, five blocks an SM: 64 take 34.7 and 32.3 us.)
    const int half = p.rot / 2;
    const int vectors = (p.heads[0] + p.heads[1]) * (layout == OQ_ROPE_HALF ? half : p.rot) /
                        Vec<E>::n;
    int tokens = kThreads * (layout == OQ_ROPE_HALF ? ahead<true>() : ahead<false>()) / vectors;
    if (tokens > kThreads / half)
        tokens = kThreads / half;
    if (tokens > p.T / (2 * num_sms))
        tokens = p.T / (2 * num_sms);
    if (tokens < 1)
        tokens = 1;
    const dim3 grid((p.T - 1) / tokens + 1);             // (T may be the largest int)
    const size_t smem = (size_t)tokens * half * sizeof(float2);
    constexpr int V = Vec<E>::n;
    const Divide turned((layout == OQ_ROPE_HALF ? half : p.rot) / V);
    const Divide copied(p.d > p.rot ? (p.d - p.rot) / V : 1), heads(p.heads[0] + p.heads[1]);
    if (layout == OQ_ROPE_HALF)
        return launch_pdl(rope_kernel<E, true>, grid, dim3(kThreads), smem, st, p, tokens, turned,
                          copied, heads);
    return launch_pdl(rope_kernel<E, false>, grid, dim3(kThreads), smem, st, p, tokens, turned,
                      copied, heads);
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, int dtype, int layout, cudaStream_t st, int num_sms,
                        std::string *why) {
    *why = "oq_apply_rope: launch";
    if (dtype == OQ_F32)
        return run<float>(p, layout, st, num_sms);
    if (dtype == OQ_BF16)
        return run<__nv_bfloat16>(p, layout, st, num_sms);
    return run<__half>(p, layout, st, num_sms);
}

}  // namespace oq
