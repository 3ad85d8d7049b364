// rope.cu -- rotary positions of queries and keys.
//
// Pair (a, b) of a head at position t becomes m (a cos - b sin, a sin + b cos) with the angle
// t * freq_i; the gradient goes back through the transpose, the same with -sin.  Bound by memory:
// each element is read and written once, 16 bytes at a time, and a block forms the cosines of its
// tokens once for all their heads.  Angles are taken in fp64 turns (t * freq / 2 pi minus its
// nearest integer), since an fp32 product at position 1e5 is already off by 1e-2 radians; the
// cosine itself is fp32 (sincospif of the reduced turns).
#include "kv_internal.h"
#include "kv_ops.cuh"

namespace oq {
namespace {

using namespace kvops;

constexpr int kThreads = 256;

template <class E, bool HALF>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p, int tokens_a_block) {
    extern __shared__ float2 cs[];                       // [tokens][rot / 2] (cos, sin)
    pdl_trigger();
    constexpr int V = Vec<E>::n;
    const int half = p.rot / 2;
    const int t0 = blockIdx.x * tokens_a_block;
    const int nt = min(tokens_a_block, p.T - t0);
    pdl_wait();
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const double turn = (double)p.pos[t0 + i / half] * p.turns[i % half];
        float s, c;
        sincospif(2.0f * (float)(turn - rint(turn)), &s, &c);
        cs[i] = make_float2(p.amplitude * c, p.inverse ? -p.amplitude * s : p.amplitude * s);
    }
    __syncthreads();
    // a head's work: HALF: half / V pairs of vectors, else rot / V vectors; then the rest copied
    const int turned = HALF ? half / V : p.rot / V;
    const int a_head = turned + (p.d - p.rot) / V;
    const int a_token = (p.heads[0] + p.heads[1]) * a_head;
    for (int i = threadIdx.x; i < nt * a_token; i += kThreads) {
        const int t = i / a_token, r = i - t * a_token;
        int head = r / a_head;
        const int j = r - head * a_head;
        const int w = head >= p.heads[0];
        head -= w ? p.heads[0] : 0;
        const long long tok = t0 + t;
        const E *x = static_cast<const E *>(p.x[w]) + tok * p.x_stride[w] + head * p.d;
        E *y = static_cast<E *>(p.y[w]) + tok * p.y_stride[w] + head * p.d;
        const float2 *a = cs + t * half;
        if (j >= turned) {
            const int at = p.rot + (j - turned) * V;
            if (x != y) {
                Vec<E> v;
                v.load(x + at);
                v.store(y + at);
            }
        } else if (HALF) {
            Vec<E> u, v;
            u.load(x + j * V);
            v.load(x + half + j * V);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float2 q = a[j * V + e];
                const float f = to_f32(u.e[e]), g = to_f32(v.e[e]);
                u.e[e] = from_f32<E>(f * q.x - g * q.y);
                v.e[e] = from_f32<E>(f * q.y + g * q.x);
            }
            u.store(y + j * V);
            v.store(y + half + j * V);
        } else {
            Vec<E> u;
            u.load(x + j * V);
#pragma unroll
            for (int e = 0; e < V; e += 2) {
                const float2 q = a[(j * V + e) / 2];
                const float f = to_f32(u.e[e]), g = to_f32(u.e[e + 1]);
                u.e[e] = from_f32<E>(f * q.x - g * q.y);
                u.e[e + 1] = from_f32<E>(f * q.y + g * q.x);
            }
            u.store(y + j * V);
        }
    }
}

template <class E>
cudaError_t run(const RopeParams &p, int layout, cudaStream_t st, int num_sms) {
    // as many tokens a block as its threads have angles for, fewer while that leaves SMs idle
    const int half = p.rot / 2;
    int tokens = kThreads / half;
    if (tokens > p.T / (2 * num_sms))
        tokens = p.T / (2 * num_sms);
    if (tokens < 1)
        tokens = 1;
    const dim3 grid((p.T + tokens - 1) / tokens);
    const size_t smem = (size_t)tokens * half * sizeof(float2);
    if (layout == OQ_ROPE_HALF)
        return launch_pdl(rope_kernel<E, true>, grid, dim3(kThreads), smem, st, p, tokens);
    return launch_pdl(rope_kernel<E, false>, grid, dim3(kThreads), smem, st, p, tokens);
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
