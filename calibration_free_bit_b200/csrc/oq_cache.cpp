// oq_cache.cpp -- host side of the rotary positions and the quantised key/value cache: the calls
// oq_build_rope .. oq_kv_attend of include/oq.h (argument checks, tables, launches).
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "kv_internal.h"
#include "oq_handles.h"

using namespace oq::host;

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;
constexpr double kLog2e = 1.4426950408889634073599246810019;

int elem_size(int dtype) { return dtype == OQ_F32 ? 4 : 2; }

// Rows [tokens, heads, d] of a tensor: base and token stride must keep 16-byte vectors aligned.
int check_rows(const char *who, const char *name, const void *p, long long stride, int dtype) {
    if (!p)
        return fail(OQ_EINVAL, "%s: %s is NULL", who, name);
    if (!aligned16(p) || stride < 0 || (stride * elem_size(dtype)) % 16 != 0)
        return fail(OQ_EINVAL, "%s: %s must be 16-byte aligned, with a token stride (%lld "
                               "elements) that is a non-negative multiple of 16 bytes", who, name,
                    stride);
    return OQ_OK;
}

// The same for a tensor that is written: tokens must not overlap.
int check_out_rows(const char *who, const char *name, const void *p, long long stride, int dtype,
                   long long row) {
    const int rc = check_rows(who, name, p, stride, dtype);
    if (rc != OQ_OK)
        return rc;
    if (stride < row)
        return fail(OQ_EINVAL, "%s: %s has a token stride of %lld elements, less than its "
                               "heads * d = %lld", who, name, stride, row);
    return OQ_OK;
}

int check_cache(const char *who, const oq_rpbh *r, const oq_codebook *c, const oq_kv_cache *cache,
                oq::KvView *v) {
    if (!r || !c || !cache)
        return fail(OQ_EINVAL, "%s: null handle or cache", who);
    if (cache->d != 128 && cache->d != 256)
        return fail(OQ_EINVAL, "%s: head dimension %d (128 or 256)", who, cache->d);
    if (r->d != cache->d || c->d != cache->d)
        return fail(OQ_EINVAL, "%s: the cache has d = %d but the rotation has d = %d and the "
                               "codebook d = %d", who, cache->d, r->d, c->d);
    if (c->bits != cache->bits)
        return fail(OQ_EINVAL, "%s: the cache has %d-bit codes but the codebook %d bits", who,
                    cache->bits, c->bits);
    if (cache->page_size < 16 || cache->page_size > 1024 ||
        (cache->page_size & (cache->page_size - 1)) != 0)
        return fail(OQ_EINVAL, "%s: page_size = %d must be a power of two in [16, 1024]", who,
                    cache->page_size);
    if (cache->kv_heads < 1 || cache->kv_heads > OQ_KV_MAX_HEADS)
        return fail(OQ_EINVAL, "%s: kv_heads = %d not in [1, %d]", who, cache->kv_heads,
                    OQ_KV_MAX_HEADS);
    if (cache->num_pages < 1 || cache->num_pages > 0x7fffffffll)
        return fail(OQ_EINVAL, "%s: num_pages = %lld not in [1, 2^31)", who, cache->num_pages);
    if (!cache->k_codes || !cache->v_codes || !cache->k_norms || !cache->v_norms)
        return fail(OQ_EINVAL, "%s: null cache pointer", who);
    if (!aligned16(cache->k_codes) || !aligned16(cache->v_codes) || !aligned16(cache->k_norms) ||
        !aligned16(cache->v_norms))
        return fail(OQ_EINVAL, "%s: the cache's arrays must be 16-byte aligned", who);
    v->codes[0] = cache->k_codes;
    v->codes[1] = cache->v_codes;
    v->norms[0] = cache->k_norms;
    v->norms[1] = cache->v_norms;
    v->pages = cache->num_pages;
    v->page_log2 = 0;
    while ((1 << v->page_log2) < cache->page_size)
        ++v->page_log2;
    v->kv_heads = cache->kv_heads;
    v->d = cache->d;
    v->bits = cache->bits;
    v->row_bytes = cache->d * cache->bits / 8;
    return OQ_OK;
}

// (tiles of 128 rows are counted in 32 bits; rows may be one row for all tokens, so memory is no limit)
int check_tokens(const char *who, int T, int heads) {
    if (T < 0 || (long long)T * heads > 1ll << 36)
        return fail(OQ_EINVAL, "%s: T = %d tokens of %d heads: negative, or over 2^36 rows", who, T,
                    heads);
    return OQ_OK;
}

int check_slots(const char *who, const int64_t *slots) {
    if (!slots || (reinterpret_cast<uintptr_t>(slots) & 7u))
        return fail(OQ_EINVAL, "%s: slots must be a non-null, 8-byte aligned pointer", who);
    return OQ_OK;
}

enum { RMAT_BF16 = 0, RMAT_F16 = 1, RMAT_F16_T = 2 };

// sqrt(h) R (entries +-1 and 0) on the current device, as the K-major, 128-byte-swizzled operand
// that kv_tc.cu copies into shared memory: row n has elements k = 0 .. d-1 in 64-wide atoms of d
// rows of 128 bytes, 16-byte chunk c of a row at chunk c ^ (n % 8).  R[i][perm[j]] = sign[j]
// (-1)^popcount(i & j) for i, j in one block.
int rotation_matrix(oq_rpbh *r, int which, int dev, const void **out) {
    {
        std::lock_guard<std::mutex> lk(r->mu);
        if (r->rmat[which].empty()) {
            const int d = r->d, h = r->h;
            const uint16_t one = which == RMAT_BF16 ? 0x3F80 : 0x3C00;
            std::vector<uint16_t> m((size_t)d * d, 0);
            for (int i = 0; i < d; ++i)
                for (int j = i / h * h; j < i / h * h + h; ++j) {
                    const bool neg = (__builtin_popcount(i & j & (h - 1)) & 1) ^ (r->sign[j] < 0);
                    const int n = which == RMAT_F16_T ? r->perm[j] : i;
                    const int k = which == RMAT_F16_T ? i : r->perm[j];
                    const size_t at = (size_t)(k >> 6) * d * 64 + (size_t)n * 64 +
                                      ((((k >> 3) & 7) ^ (n & 7)) << 3) + (k & 7);
                    m[at] = (uint16_t)(one | (neg ? 0x8000 : 0));
                }
            r->rmat[which] = std::move(m);
        }
    }
    const int rc = upload(r->mu, &r->dev_rmat[which][dev], r->rmat[which], "upload rotation matrix");
    *out = r->dev_rmat[which][dev];
    return rc;
}

int upload_ent(oq_rpbh *r, int dev) {
    return upload(r->mu, &r->dev_ent16[dev], r->ent16, "upload rotation entries");
}

// The fp16 decode table of the cache's kernels: 32-bit words of two centroids.
//   bits 2: entry e (a byte, four codes) = two words; bits 3, 4: entry e (two codes) = one word,
//   the lower code in the low half; bits 6, 8: entry e (one code) in the low half, what fp16 leaves
//   of it in the high one.
// The centroids are multiplied by kv_alpha in [1, 2) before they are rounded to fp16, and the
// kernels divide by it in fp32: of 4096 factors the one whose rounded centroids are nearest (cells
// weighted by the mass that the quantizer gives them).  At 4 bits that takes the rounding from
// 2.8e-4 of a centroid (rms) to about 0.5e-4, at 2 and 3 bits to below 1e-5.
void build_kv_lut(oq_codebook *cb) {
    const int L = 1 << cb->bits;
    auto value = [](uint16_t h) {
        const int e = (h >> 10) & 31;
        const double m = std::ldexp(1024.0 + (h & 1023), e - 25);
        return (h & 0x8000) ? -m : m;
    };
    std::vector<double> mass(L);
    for (int i = 0; i < L; ++i) {                 // N(0, 1) density times the cell's width
        const double lo = i ? cb->t[i - 1] : cb->c[0] - (cb->t[0] - cb->c[0]);
        const double hi = i + 1 < L ? cb->t[i] : 2.0 * cb->c[L - 1] - cb->t[L - 2];
        mass[i] = std::exp(-0.5 * cb->c[i] * cb->c[i]) * (hi - lo);
    }
    // x to the 11 significant bits of fp16 (all of a c is in its normal range), to nearest even
    auto rounded = [](double x) {
        uint64_t u;
        std::memcpy(&u, &x, 8);
        u = (u + ((1ull << 41) - 1) + ((u >> 42) & 1)) & ~((1ull << 42) - 1);
        std::memcpy(&x, &u, 8);
        return x;
    };
    double best = -1.0;
    const int tries = L <= 16 ? 4096 : 4096 / L;  // of many centroids all factors leave about the same
    for (int k = 0; k < tries; ++k) {
        const double a = 1.0 + (double)k / tries;
        double err = 0.0;
        for (int i = L / 2; i < L; ++i) {
            const double d = rounded(a * cb->c[i]) / a - cb->c[i];
            err += mass[i] * d * d;
        }
        if (best < 0.0 || err < best) {
            best = err;
            cb->kv_alpha = a;
        }
    }
    uint16_t lut[256];
    for (int i = 0; i < L; ++i)
        lut[i] = to_half_bits(cb->kv_alpha * cb->c[i]);
    std::vector<uint32_t> out;
    const int b = cb->bits;
    const int entries = b == 6 || b == 3 ? 64 : 256;
    for (int e = 0; e < entries; ++e) {
        if (b == 2)
            for (int k = 0; k < 2; ++k)
                out.push_back(lut[(e >> (4 * k)) & 3] |
                              (uint32_t)lut[(e >> (4 * k + 2)) & 3] << 16);
        else if (b <= 4)
            out.push_back(lut[e & (L - 1)] | (uint32_t)lut[e >> b] << 16);
        else                                      // and what fp16 leaves of it
            out.push_back(lut[e] | (uint32_t)to_half_bits(cb->kv_alpha * cb->c[e] - value(lut[e])) << 16);
    }
    cb->kv_lut = std::move(out);
}

// The decode table on the current device, made at a codebook's first use with a cache (most
// codebooks never see one, and the search for kv_alpha takes longer than the rest of them).
int decode_table(oq_codebook *cb, int dev) {
    {
        std::lock_guard<std::mutex> lk(cb->mu);
        if (cb->kv_lut.empty())
            build_kv_lut(cb);
    }
    return upload(cb->mu, &cb->dev_kv_lut[dev], cb->kv_lut, "upload decode table");
}

}  // namespace

extern "C" {

int oq_build_rope(int rot_dim, int layout, double theta, int scaling, double factor,
                  int original_len, oq_rope **out) {
    const char *who = "oq_build_rope";
    if (!out)
        return fail(OQ_EINVAL, "%s: out is NULL", who);
    *out = nullptr;
    if (rot_dim < 16 || rot_dim > 512 || rot_dim % 16 != 0)
        return fail(OQ_EINVAL, "%s: rot_dim = %d must be a multiple of 16 in [16, 512]", who,
                    rot_dim);
    if (layout != OQ_ROPE_HALF && layout != OQ_ROPE_INTERLEAVED)
        return fail(OQ_EINVAL, "%s: layout = %d (OQ_ROPE_HALF or OQ_ROPE_INTERLEAVED)", who,
                    layout);
    if (!(theta > 1.0) || !std::isfinite(theta))
        return fail(OQ_EINVAL, "%s: theta must be finite and above 1", who);
    if (scaling < OQ_ROPE_PLAIN || scaling > OQ_ROPE_YARN)
        return fail(OQ_EINVAL, "%s: scaling = %d (OQ_ROPE_PLAIN .. OQ_ROPE_YARN)", who, scaling);
    if (scaling != OQ_ROPE_PLAIN && !(factor >= 1.0 && std::isfinite(factor)))
        return fail(OQ_EINVAL, "%s: factor must be finite and at least 1", who);
    if (scaling == OQ_ROPE_YARN && original_len < 1)
        return fail(OQ_EINVAL, "%s: original_len = %d must be positive", who, original_len);
    oq_rope *r = new (std::nothrow) oq_rope;
    if (!r)
        return fail(OQ_ENOMEM, "%s: out of host memory", who);
    r->rot = rot_dim;
    r->layout = layout;
    const int half = rot_dim / 2;
    const double base =
        scaling == OQ_ROPE_NTK ? theta * std::pow(factor, (double)rot_dim / (rot_dim - 2)) : theta;
    r->freq.resize(half);
    for (int i = 0; i < half; ++i)
        r->freq[i] = std::pow(base, -2.0 * i / rot_dim);
    if (scaling == OQ_ROPE_LINEAR)
        for (double &f : r->freq)
            f /= factor;
    if (scaling == OQ_ROPE_YARN) {
        // the pair that makes `turns` turns over the original length
        auto pair_at = [&](double turns) {
            return rot_dim * std::log(original_len / (turns * kTwoPi)) / (2.0 * std::log(theta));
        };
        const double lo = std::max(std::floor(pair_at(32.0)), 0.0);
        const double hi = std::min(std::ceil(pair_at(1.0)), rot_dim - 1.0);
        for (int i = 0; i < half; ++i) {
            const double ramp = std::min(std::max((i - lo) / std::max(hi - lo, 1e-3), 0.0), 1.0);
            r->freq[i] = r->freq[i] / factor * ramp + r->freq[i] * (1.0 - ramp);
        }
        r->amplitude = 0.1 * std::log(factor) + 1.0;
    }
    r->turns.resize(half);
    for (int i = 0; i < half; ++i)
        r->turns[i] = r->freq[i] / kTwoPi;
    *out = r;
    return OQ_OK;
}

int oq_rope_values(const oq_rope *r, double *freq, double *amplitude) {
    if (!r)
        return fail(OQ_EINVAL, "oq_rope_values: null handle");
    if (freq)
        std::memcpy(freq, r->freq.data(), sizeof(double) * r->freq.size());
    if (amplitude)
        *amplitude = r->amplitude;
    return OQ_OK;
}

void oq_free_rope(oq_rope *r) {
    if (!r)
        return;
    int cur = -1;
    cudaGetDevice(&cur);
    for (int dev = 0; dev < oq::kMaxDevices; ++dev)
        if (r->dev_turns[dev]) {
            cudaSetDevice(dev);
            cudaFree(r->dev_turns[dev]);
        }
    if (cur >= 0)
        cudaSetDevice(cur);
    delete r;
}

int oq_apply_rope(const oq_rope *r, const void *x, long long x_stride, void *y, long long y_stride,
                  int heads, const void *k, long long k_stride, void *ky, long long ky_stride,
                  int k_heads, int dtype, int T, int d, const int64_t *positions, int inverse,
                  void *stream) {
    const char *who = "oq_apply_rope";
    if (!r)
        return fail(OQ_EINVAL, "%s: null handle", who);
    if (dtype != OQ_F32 && dtype != OQ_BF16 && dtype != OQ_F16)
        return fail(OQ_EINVAL, "%s: dtype must be OQ_F32, OQ_BF16 or OQ_F16", who);
    if (d < r->rot || d > 1024 || d % 16 != 0)
        return fail(OQ_EINVAL, "%s: d = %d must be a multiple of 16 from rot_dim = %d to 1024",
                    who, d, r->rot);
    if (T < 0)
        return fail(OQ_EINVAL, "%s: negative row count %d", who, T);
    oq::RopeParams p{};
    p.x[0] = x, p.y[0] = y, p.x_stride[0] = x_stride, p.y_stride[0] = y_stride, p.heads[0] = heads;
    if (k)
        p.x[1] = k, p.y[1] = ky, p.x_stride[1] = k_stride, p.y_stride[1] = ky_stride,
        p.heads[1] = k_heads;
    for (int i = 0; i < (k ? 2 : 1); ++i)
        if (p.heads[i] < 1 || p.heads[i] > OQ_KV_MAX_HEADS)
            return fail(OQ_EINVAL, "%s: %d heads, not in [1, %d]", who, p.heads[i],
                        OQ_KV_MAX_HEADS);
    if (T == 0)
        return OQ_OK;
    if (!positions || (reinterpret_cast<uintptr_t>(positions) & 7u))
        return fail(OQ_EINVAL, "%s: positions must be a non-null, 8-byte aligned pointer", who);
    for (int i = 0; i < (k ? 2 : 1); ++i) {
        int rc = check_rows(who, i ? "k" : "x", p.x[i], p.x_stride[i], dtype);
        if (rc == OQ_OK)
            rc = check_out_rows(who, i ? "ky" : "y", p.y[i], p.y_stride[i], dtype,
                                (long long)p.heads[i] * d);
        if (rc != OQ_OK)
            return rc;
        if (p.x[i] == p.y[i] && p.x_stride[i] != p.y_stride[i])
            return fail(OQ_EINVAL, "%s: in place, both strides of %s must be the same", who,
                        i ? "k" : "x");
    }
    int dev;
    DeviceInfo *di;
    int rc = current_device(&dev, &di);
    if (rc != OQ_OK)
        return rc;
    oq_rope *rw = const_cast<oq_rope *>(r);
    if ((rc = upload(rw->mu, &rw->dev_turns[dev], rw->turns, "upload rotary frequencies")) != OQ_OK)
        return rc;
    p.pos = reinterpret_cast<const long long *>(positions);
    p.turns = reinterpret_cast<const double *>(rw->dev_turns[dev]);
    p.amplitude = (float)r->amplitude;
    p.T = T;
    p.d = d;
    p.rot = r->rot;
    p.inverse = inverse != 0;
    cudaStream_t st = (cudaStream_t)stream;
    std::string why;
    cudaError_t e = timed(OQ_KERNEL_ROPE, st, [&] {
        return oq::launch_rope(p, dtype, r->layout, st, di->sms, &why);
    });
    return e == cudaSuccess ? OQ_OK : fail_cuda(e, why.c_str());
}

int oq_kv_write(const oq_rpbh *r, const oq_codebook *c, const oq_kv_cache *cache, const void *k,
                long long k_stride, const void *v, long long v_stride, int dtype, int T,
                const int64_t *slots, void *stream) {
    const char *who = "oq_kv_write";
    oq::KvWriteParams p{};
    int rc = check_cache(who, r, c, cache, &p.c);
    if (rc != OQ_OK)
        return rc;
    if (dtype != OQ_F32 && dtype != OQ_BF16 && dtype != OQ_F16)
        return fail(OQ_EINVAL, "%s: dtype must be OQ_F32, OQ_BF16 or OQ_F16", who);
    if ((rc = check_tokens(who, T, cache->kv_heads)) != OQ_OK)
        return rc;
    if (T == 0)
        return OQ_OK;
    if ((rc = check_rows(who, "k", k, k_stride, dtype)) != OQ_OK ||
        (rc = check_rows(who, "v", v, v_stride, dtype)) != OQ_OK ||
        (rc = check_slots(who, slots)) != OQ_OK)
        return rc;
    int dev;
    DeviceInfo *di;
    if ((rc = current_device(&dev, &di)) != OQ_OK)
        return rc;
    oq_rpbh *rw = const_cast<oq_rpbh *>(r);
    oq_codebook *cw = const_cast<oq_codebook *>(c);
    if ((rc = upload_ent(rw, dev)) != OQ_OK ||
        (rc = upload(cw->mu, &cw->dev_tbl[dev], cw->tbl_img, "upload quantizer table")) != OQ_OK ||
        (rc = upload(cw->mu, &cw->dev_cent32[dev], cw->cent32, "upload centroids")) != OQ_OK)
        return rc;
    if (dtype != OQ_F32 &&
        (rc = rotation_matrix(rw, dtype == OQ_BF16 ? RMAT_BF16 : RMAT_F16, dev, &p.r_img)) != OQ_OK)
        return rc;
    p.x[0] = k;
    p.x[1] = v;
    p.x_stride[0] = k_stride;
    p.x_stride[1] = v_stride;
    p.slots = reinterpret_cast<const long long *>(slots);
    p.T = T;
    p.h = r->h;
    p.ent = reinterpret_cast<const uint16_t *>(rw->dev_ent16[dev]);
    p.tbl = cw->dev_tbl[dev];
    p.tbl_copies = c->bits <= 4 ? 32 : 1;
    p.tbl_words = (int)cw->tbl_img.size();
    p.bounds = reinterpret_cast<const float *>(cw->dev_cent32[dev]) + (1 << c->bits);
    p.unit = std::sqrt((double)r->d / r->h);
    p.wide = p.c.row_bytes % 32 == 0 &&
             ((reinterpret_cast<uintptr_t>(cache->k_codes) |
               reinterpret_cast<uintptr_t>(cache->v_codes)) & 31u) == 0;
    p.eps = 1e-8f;
    p.K = (float)(std::sqrt((double)r->d / r->h) / (c->G * c->delta));
    p.G = c->G;
    p.F = c->F;
    cudaStream_t st = (cudaStream_t)stream;
    std::string why;
    cudaError_t e = timed(OQ_KERNEL_KV_WRITE, st, [&] {
        return oq::launch_kv_write(p, dtype, st, di->sms, &why);
    });
    return e == cudaSuccess ? OQ_OK : fail_cuda(e, why.c_str());
}

int oq_kv_read(const oq_rpbh *r, const oq_codebook *c, const oq_kv_cache *cache,
               const int64_t *slots, int T, void *k, long long k_stride, void *v,
               long long v_stride, int dtype, void *stream) {
    const char *who = "oq_kv_read";
    oq::KvReadParams p{};
    int rc = check_cache(who, r, c, cache, &p.c);
    if (rc != OQ_OK)
        return rc;
    if (dtype != OQ_F32 && dtype != OQ_BF16 && dtype != OQ_F16)
        return fail(OQ_EINVAL, "%s: dtype must be OQ_F32, OQ_BF16 or OQ_F16", who);
    if ((rc = check_tokens(who, T, cache->kv_heads)) != OQ_OK)
        return rc;
    if (T == 0)
        return OQ_OK;
    const long long row = (long long)cache->kv_heads * cache->d;
    if ((rc = check_out_rows(who, "k", k, k_stride, dtype, row)) != OQ_OK ||
        (rc = check_out_rows(who, "v", v, v_stride, dtype, row)) != OQ_OK ||
        (rc = check_slots(who, slots)) != OQ_OK)
        return rc;
    int dev;
    DeviceInfo *di;
    if ((rc = current_device(&dev, &di)) != OQ_OK)
        return rc;
    oq_rpbh *rw = const_cast<oq_rpbh *>(r);
    oq_codebook *cw = const_cast<oq_codebook *>(c);
    if ((rc = upload_ent(rw, dev)) != OQ_OK ||
        (rc = upload(cw->mu, &cw->dev_cent32[dev], cw->cent32, "upload centroids")) != OQ_OK)
        return rc;
    if (dtype != OQ_F32 &&
        ((rc = rotation_matrix(rw, RMAT_F16_T, dev, &p.r_img)) != OQ_OK ||
         (rc = decode_table(cw, dev)) != OQ_OK))
        return rc;
    p.lut = cw->dev_kv_lut[dev];
    p.alpha_inv = dtype == OQ_F32 ? 1.f : (float)(1.0 / c->kv_alpha);   // (rows kernel: no table)
    p.y[0] = k;
    p.y[1] = v;
    p.y_stride[0] = k_stride;
    p.y_stride[1] = v_stride;
    p.slots = reinterpret_cast<const long long *>(slots);
    p.T = T;
    p.h = r->h;
    p.ent = reinterpret_cast<const uint16_t *>(rw->dev_ent16[dev]);
    p.cent = reinterpret_cast<const float *>(cw->dev_cent32[dev]);
    p.scale = (float)(1.0 / std::sqrt((double)r->d * r->h));
    cudaStream_t st = (cudaStream_t)stream;
    std::string why;
    cudaError_t e = timed(OQ_KERNEL_KV_READ, st, [&] {
        return oq::launch_kv_read(p, dtype, st, di->sms, &why);
    });
    return e == cudaSuccess ? OQ_OK : fail_cuda(e, why.c_str());
}

int oq_kv_attend(const oq_rpbh *r, const oq_codebook *c, const oq_kv_cache *cache, const void *q,
                 long long q_stride, void *out, long long out_stride, int dtype, int q_rows,
                 int q_heads, const int32_t *q_start, const int32_t *prefix, int B, int max_nodes,
                 const int32_t *page_table, int table_width, const int64_t *tree_mask,
                 double scale, void *stream) {
    const char *who = "oq_kv_attend";
    oq::KvAttendParams p{};
    int rc = check_cache(who, r, c, cache, &p.c);
    if (rc != OQ_OK)
        return rc;
    if (dtype != OQ_BF16 && dtype != OQ_F16)
        return fail(OQ_EINVAL, "%s: dtype must be OQ_BF16 or OQ_F16", who);
    if (q_heads < 1 || q_heads > OQ_KV_MAX_HEADS || q_heads % cache->kv_heads != 0)
        return fail(OQ_EINVAL, "%s: q_heads = %d must be a multiple of kv_heads = %d, at most %d",
                    who, q_heads, cache->kv_heads, OQ_KV_MAX_HEADS);
    if (q_rows < 0 || B < 0 || B > 65535)
        return fail(OQ_EINVAL, "%s: q_rows = %d and B = %d must be non-negative, B at most 65535",
                    who, q_rows, B);
    if (max_nodes < 1 || max_nodes > OQ_KV_MAX_NODES)
        return fail(OQ_EINVAL, "%s: max_nodes = %d not in [1, %d]", who, max_nodes,
                    OQ_KV_MAX_NODES);
    // (tiles of up to 128 tokens are counted in 32 bits)
    if (table_width < 1 || ((long long)table_width << p.c.page_log2) > 0x7fffff00ll)
        return fail(OQ_EINVAL, "%s: table_width = %d must be positive, and hold at most 2^31 - 256 "
                               "tokens", who, table_width);
    if (!(scale > 0.0) || !std::isfinite((float)(scale * kLog2e)))
        return fail(OQ_EINVAL, "%s: scale must be positive and, times log2(e), finite in fp32", who);
    if (q_rows == 0 || B == 0)
        return OQ_OK;
    if ((rc = check_rows(who, "q", q, q_stride, dtype)) != OQ_OK ||
        (rc = check_out_rows(who, "out", out, out_stride, dtype, (long long)q_heads * cache->d)) !=
            OQ_OK)
        return rc;
    if (q == out && q_stride != out_stride)
        return fail(OQ_EINVAL, "%s: in place, both strides must be the same", who);
    if (!q_start || !prefix || !page_table)
        return fail(OQ_EINVAL, "%s: null q_start, prefix or page_table", who);
    if (((reinterpret_cast<uintptr_t>(q_start) | reinterpret_cast<uintptr_t>(prefix) |
          reinterpret_cast<uintptr_t>(page_table)) & 3u) ||
        (reinterpret_cast<uintptr_t>(tree_mask) & 7u))
        return fail(OQ_EINVAL, "%s: q_start, prefix and page_table must be 4-byte aligned, "
                               "tree_mask 8-byte", who);
    int dev;
    DeviceInfo *di;
    if ((rc = current_device(&dev, &di)) != OQ_OK)
        return rc;
    oq_rpbh *rw = const_cast<oq_rpbh *>(r);
    oq_codebook *cw = const_cast<oq_codebook *>(c);
    if ((rc = upload_ent(rw, dev)) != OQ_OK ||
        (rc = decode_table(cw, dev)) != OQ_OK)
        return rc;
    p.q = q;
    p.out = out;
    p.q_stride = q_stride;
    p.out_stride = out_stride;
    p.q_heads = q_heads;
    p.group = q_heads / cache->kv_heads;
    p.q_rows = q_rows;
    p.q_start = q_start;
    p.prefix = prefix;
    p.table = page_table;
    p.mask = reinterpret_cast<const long long *>(tree_mask);
    p.B = B;
    p.table_width = table_width;
    p.max_nodes = max_nodes;
    p.ent = reinterpret_cast<const uint16_t *>(rw->dev_ent16[dev]);
    p.lut = cw->dev_kv_lut[dev];
    p.h = r->h;
    const double unit = 1.0 / (std::sqrt((double)r->d * r->h) * c->kv_alpha);
    p.qk_scale = (float)(scale * kLog2e * unit);
    p.o_scale = (float)unit;
    cudaStream_t st = (cudaStream_t)stream;
    std::string why;
    if (p.c.d == 128 && dtype == OQ_BF16 &&
        (rc = rotation_matrix(rw, RMAT_BF16, dev, &p.r_img)) != OQ_OK)
        return rc;
    void *space = nullptr;
    const size_t need = oq::kv_attend_space(p, dtype, di->sms);
    cudaError_t e = cudaSuccess;
    if (need > 0) {
        cudaMemPool_t pool = device_pool(dev, di, &rc);
        if (!pool)
            return rc;
        e = cudaMallocFromPoolAsync(&space, need, pool, st);
        if (e != cudaSuccess)
            return fail_cuda(e, "oq_kv_attend: workspace allocation");
    }
    e = timed(OQ_KERNEL_KV_ATTEND, st, [&] {
        return oq::launch_kv_attend(p, space, dtype, st, di->sms, &why);
    });
    const cudaError_t e2 = space ? cudaFreeAsync(space, st) : cudaSuccess;
    if (e != cudaSuccess)
        return fail_cuda(e, why.c_str());
    if (e2 != cudaSuccess)
        return fail_cuda(e2, "oq_kv_attend: workspace release");
    return OQ_OK;
}

}  // extern "C"
