// C-ABI of the operators of a layer in 8 bits: argument checks and launches of
// quantisation, norm and product, which keep no state, and the plan of the
// 8-bit copies of many weights.
#include "../../include/shampoo.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "fp8.hpp"

using namespace shampoo;

namespace {

constexpr int64_t kMaxSize = (int64_t)1 << 40;
constexpr int64_t kMaxTiles8 = (int64_t)1 << 24;   // workgroups of 256 threads in a launch

int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
int64_t blocks_of(int64_t cols) { return (cols + kBlock8 - 1) / kBlock8; }
int status_of(hipError_t e) { return e == hipSuccess ? SHAMPOO_OK : SHAMPOO_E_HIP; }
bool size_ok(int64_t n) { return n >= 0 && n <= kMaxSize; }
bool type_ok(int t) { return t >= SHAMPOO_F32 && t <= SHAMPOO_F16; }
int64_t bytes_of(int t) { return t == SHAMPOO_F32 ? 4 : 2; }
bool aligned_to(const void* p, uint64_t a) { return reinterpret_cast<uint64_t>(p) % a == 0; }

// Whether fewer than 2^24 tiles cover rows x cols.
bool tiles_ok(int64_t rows, int64_t cols, int64_t tr, int64_t tc) {
    return (double)((rows + tr - 1) / tr) * (double)((cols + tc - 1) / tc) < (double)kMaxTiles8;
}

// Rows of memory: what a matrix occupies.
struct Area {
    uint64_t base;
    int64_t rows, width, pitch;   // bytes
    bool empty() const { return rows <= 0 || width <= 0; }
    uint64_t end() const { return base + (uint64_t)((rows - 1) * pitch + width); }
};
// Whether two areas share a byte.  Ones side by side in the rows of one buffer
// do not; beyond that, interleaved areas of different pitches count as
// overlapping.
bool overlap(const Area& a, const Area& b) {
    if (a.empty() || b.empty() || a.end() <= b.base || b.end() <= a.base) return false;
    if (a.rows == 1 || b.rows == 1) {
        const int64_t pitch = a.rows == 1 ? b.pitch : a.pitch;
        if (a.rows == 1 && b.rows == 1) return true;
        const Area& one = a.rows == 1 ? a : b;
        const Area& many = a.rows == 1 ? b : a;
        const int64_t d = (int64_t)(one.base - many.base) % pitch, at = d < 0 ? d + pitch : d;
        return at < many.width || at + one.width > pitch;
    }
    if (a.pitch != b.pitch) return true;
    const int64_t d = (int64_t)(b.base - a.base) % a.pitch, at = d < 0 ? d + a.pitch : d;
    return at < a.width || at + b.width > a.pitch;
}

// Whether an area's offsets stay far inside 64 bits.
bool spans(const Area& a) { return (double)a.rows * (double)(a.pitch > a.width ? a.pitch : a.width) < 0x1p60; }

// A wide matrix: its area, and whether its address and pitch will do.
bool wide(const void* p, int type, int64_t pitch, int64_t rows, int64_t cols, Area& out) {
    if (!type_ok(type)) return false;
    const int64_t b = bytes_of(type);
    out = Area{reinterpret_cast<uint64_t>(p), rows, cols * b, pitch * b};
    if (out.empty()) return true;
    return p && aligned_to(p, b) && pitch >= 0 && pitch <= kMaxSize && (pitch >= cols || rows == 1) && spans(out);
}

// An 8-bit matrix of a given shape: two areas.
bool matrix8(const shampoo_matrix8* m, int64_t rows, int64_t cols, Area& codes, Area& scales) {
    if (m->rows != rows || m->cols != cols || m->format < SHAMPOO_E4M3 || m->format > SHAMPOO_E5M2 || m->reserved) return false;
    const int64_t width = up(cols, kBlock8);
    codes = Area{reinterpret_cast<uint64_t>(m->codes), rows, width, m->pitch};
    scales = Area{reinterpret_cast<uint64_t>(m->scales), (blocks_of(cols) + 3) / 4, 4 * rows, 4 * m->scale_pitch};
    if (codes.empty()) return true;
    return m->codes && m->scales && aligned_to(m->codes, 16) && aligned_to(m->scales, 4) && m->pitch % 16 == 0 &&
           m->pitch >= width && m->pitch <= kMaxSize && m->scale_pitch >= rows && m->scale_pitch <= kMaxSize &&
           spans(codes) && spans(scales);
}

// Whether offsets inside 256 rows of it, and of its scales, fit 32 bits.
bool rows_fit(const shampoo_matrix8* m) { return m->pitch <= (int64_t)1 << 23; }

Mat8 device_view(const shampoo_matrix8* m) {
    return Mat8{reinterpret_cast<uint64_t>(m->codes), reinterpret_cast<uint64_t>(m->scales), m->pitch, m->scale_pitch};
}
uint64_t addr(const void* p) { return reinterpret_cast<uint64_t>(p); }

// Whether an output that may stand in an input's place is that input, exactly.
bool same_place(const void* a, int64_t pa, int ta, const void* b, int64_t pb, int tb, int64_t rows) {
    return a == b && ta == tb && (pa == pb || rows == 1);
}

bool any_overlap(const Area* outs, int no, const Area* ins, int ni) {
    for (int i = 0; i < no; ++i) {
        for (int k = 0; k < ni; ++k)
            if (overlap(outs[i], ins[k])) return true;
        for (int k = 0; k < i; ++k)
            if (overlap(outs[i], outs[k])) return true;
    }
    return false;
}

}  // namespace

struct shampoo_weights8_s {
    std::vector<shampoo_weight_desc> desc;
    std::vector<QuantJob> jobs;          // addresses relative to the state until it is bound
    std::vector<QuantTile> tiles;
    shampoo_weights8_layout lay{};
    int64_t off_jobs = 0, off_tiles = 0;
    int type = 0;
    unsigned char* arena = nullptr;
    bool bound = false, weights_bound = false;
    int device = -1;
};

namespace {

bool on_device(int device) {
    int d = -1;
    return hipGetDevice(&d) == hipSuccess && d == device;
}

Mat8 placed(int64_t rows, int64_t cols, int64_t& codes, int64_t& scales) {
    Mat8 m{(uint64_t)codes, (uint64_t)scales, up(cols, kBlock8), rows};
    codes += up(rows * m.pitch, 256);
    scales += up(4 * rows * ((blocks_of(cols) + 3) / 4), 256);
    return m;
}

}  // namespace

extern "C" {

int shampoo_quantize8(const void* x, int32_t type, int64_t pitch, int64_t nrows, int64_t ncols,
                      const shampoo_matrix8* rows, const shampoo_matrix8* cols, void* stream) {
    Area in, out[4];
    int n = 0;
    if (!size_ok(nrows) || !size_ok(ncols) || (!rows && !cols)) return SHAMPOO_E_ARG;
    if (!wide(x, type, pitch, nrows, ncols, in)) return SHAMPOO_E_ARG;
    if (rows) {
        if (!matrix8(rows, nrows, ncols, out[n], out[n + 1])) return SHAMPOO_E_ARG;
        n += 2;
    }
    if (cols) {
        if (!matrix8(cols, ncols, nrows, out[n], out[n + 1])) return SHAMPOO_E_ARG;
        n += 2;
    }
    if (any_overlap(out, n, &in, 1)) return SHAMPOO_E_ARG;
    if (in.empty()) return SHAMPOO_OK;
    if (!tiles_ok(nrows, ncols, kBlock8, kBlock8)) return SHAMPOO_E_UNSUPPORTED;
    QuantJob j{};
    j.x = Wide{addr(x), pitch};
    if (rows) j.rows = device_view(rows);
    if (cols) j.cols = device_view(cols);
    j.nrows = nrows;
    j.ncols = ncols;
    return status_of(launch_quantize(type, rows ? rows->format : 0, cols ? cols->format : 0, j,
                                     static_cast<hipStream_t>(stream)));
}

int shampoo_transpose8(const shampoo_matrix8* m, const shampoo_matrix8* out, void* stream) {
    Area in[2], o[2];
    if (!m || !out || !size_ok(m->rows) || !size_ok(m->cols)) return SHAMPOO_E_ARG;
    if (!matrix8(m, m->rows, m->cols, in[0], in[1]) || !matrix8(out, m->cols, m->rows, o[0], o[1])) return SHAMPOO_E_ARG;
    if (any_overlap(o, 2, in, 2)) return SHAMPOO_E_ARG;
    if (in[0].empty()) return SHAMPOO_OK;
    if (!tiles_ok(m->rows, m->cols, kBlock8, kBlock8)) return SHAMPOO_E_UNSUPPORTED;
    QuantJob j{};
    j.src = device_view(m);
    j.cols = device_view(out);
    j.nrows = m->rows;
    j.ncols = m->cols;
    return status_of(launch_quantize(m->format == SHAMPOO_E4M3 ? SRC_E4M3 : SRC_E5M2, 0, out->format, j,
                                     static_cast<hipStream_t>(stream)));
}

int shampoo_rms_norm8(const shampoo_rms_norm_args* a, void* stream) {
    if (!a || !size_ok(a->rows) || !size_ok(a->dim) || a->dim < 1) return SHAMPOO_E_ARG;
    if (!(a->eps > 0.0 && std::isfinite(a->eps)&& a->eps >= 0x1p-120 && a->eps <= 0x1p120)) return SHAMPOO_E_ARG;
    if ((a->residual != nullptr) != (a->total != nullptr) && a->rows) return SHAMPOO_E_ARG;
    const bool res = a->residual && a->total;
    Area in[3], out[5];
    int ni = 0, no = 0;
    if (!wide(a->x, a->x_type, a->x_pitch, a->rows, a->dim, in[ni++])) return SHAMPOO_E_ARG;
    if (!wide(a->weight, a->weight_type, a->dim, a->rows ? 1 : 0, a->dim, in[ni++])) return SHAMPOO_E_ARG;
    if (res) {
        Area r, t;
        if (!wide(a->residual, a->residual_type, a->residual_pitch, a->rows, a->dim, r)) return SHAMPOO_E_ARG;
        if (!wide(a->total, a->residual_type, a->total_pitch, a->rows, a->dim, t)) return SHAMPOO_E_ARG;
        const bool over_x = same_place(a->total, a->total_pitch, a->residual_type, a->x, a->x_pitch, a->x_type, a->rows);
        const bool over_r = same_place(a->total, a->total_pitch, a->residual_type, a->residual, a->residual_pitch,
                                       a->residual_type, a->rows);
        // the sum against what it does not stand on, before the rest
        if ((!over_x && overlap(t, in[0])) || (!over_r && overlap(t, r)) || overlap(t, in[1])) return SHAMPOO_E_ARG;
        in[ni++] = r;
        out[no++] = t;
    }
    const int rest = no;
    if (a->rstd) {
        if (!aligned_to(a->rstd, 4)) return SHAMPOO_E_ARG;
        out[no++] = Area{addr(a->rstd), 1, 4 * a->rows, 4 * a->rows};
    }
    if (a->out && !wide(a->out, a->out_type, a->out_pitch, a->rows, a->dim, out[no++])) return SHAMPOO_E_ARG;
    if (a->out8) {
        if (!matrix8(a->out8, a->rows, a->dim, out[no], out[no + 1])) return SHAMPOO_E_ARG;
        no += 2;
    }
    if (!a->out && !a->out8 && a->rows) return SHAMPOO_E_ARG;
    for (int i = rest; i < no; ++i) {
        for (int k = 0; k < ni; ++k)
            if (overlap(out[i], in[k])) return SHAMPOO_E_ARG;
        for (int k = 0; k < i; ++k)
            if (overlap(out[i], out[k])) return SHAMPOO_E_ARG;
    }
    if (a->out8 && a->out8->format != SHAMPOO_E4M3) return SHAMPOO_E_UNSUPPORTED;
    if (a->rows == 0) return SHAMPOO_OK;
    if (!norm_fwd_fits(a->rows, a->dim)) return SHAMPOO_E_UNSUPPORTED;
    NormFwdArgs k{};
    k.x = Wide{addr(a->x), a->x_pitch};
    if (res) {
        k.res = Wide{addr(a->residual), a->residual_pitch};
        k.total = Wide{addr(a->total), a->total_pitch};
    }
    k.out = Wide{addr(a->out), a->out_pitch};
    if (a->out8) k.out8 = device_view(a->out8);
    k.w = a->weight;
    k.rstd = a->rstd;
    k.rows = a->rows;
    k.dim = a->dim;
    k.eps = a->eps;
    k.w_type = a->weight_type;
    k.out_type = a->out_type;
    return status_of(launch_norm_fwd(a->x_type, res ? a->residual_type : -1, k, static_cast<hipStream_t>(stream)));
}

int shampoo_rms_norm8_backward_workspace(int64_t rows, int64_t dim, size_t* bytes) {
    if (!bytes || !size_ok(rows) || !size_ok(dim) || dim < 1) return SHAMPOO_E_ARG;
    *bytes = (size_t)norm_bwd_slots(rows, dim) * (size_t)dim * 4;
    return SHAMPOO_OK;
}

int shampoo_rms_norm8_backward(const shampoo_rms_norm_grad_args* a, void* workspace, size_t bytes, void* stream) {
    if (!a || !size_ok(a->rows) || !size_ok(a->dim) || a->dim < 1 || a->accumulate < 0 || a->accumulate > 1) return SHAMPOO_E_ARG;
    Area in[5], out[3];
    int ni = 0, no = 0;
    Area g, z, add{}, dz;
    if (!wide(a->grad, a->grad_type, a->grad_pitch, a->rows, a->dim, g)) return SHAMPOO_E_ARG;
    if (!wide(a->z, a->z_type, a->z_pitch, a->rows, a->dim, z)) return SHAMPOO_E_ARG;
    if (a->add && !wide(a->add, a->z_type, a->add_pitch, a->rows, a->dim, add)) return SHAMPOO_E_ARG;
    if (!wide(a->dz, a->z_type, a->dz_pitch, a->rows, a->dim, dz)) return SHAMPOO_E_ARG;
    if (!wide(a->weight, a->weight_type, a->dim, a->rows ? 1 : 0, a->dim, in[ni++])) return SHAMPOO_E_ARG;
    if (a->rows && (!a->rstd || !aligned_to(a->rstd, 4))) return SHAMPOO_E_ARG;
    if (!aligned_to(a->dw, 4)) return SHAMPOO_E_ARG;
    in[ni++] = Area{addr(a->rstd), 1, 4 * a->rows, 4 * a->rows};
    const auto on = [&](const void* p, int64_t pitch, int type) {
        return same_place(a->dz, a->dz_pitch, a->z_type, p, pitch, type, a->rows);
    };
    if ((!on(a->grad, a->grad_pitch, a->grad_type) && overlap(dz, g)) || (!on(a->z, a->z_pitch, a->z_type) && overlap(dz, z)) ||
        (a->add && !on(a->add, a->add_pitch, a->z_type) && overlap(dz, add)) || overlap(dz, in[0]) || overlap(dz, in[1]))
        return SHAMPOO_E_ARG;
    in[ni++] = g;
    in[ni++] = z;
    if (a->add) in[ni++] = add;
    if (a->dw) out[no++] = Area{addr(a->dw), 1, 4 * a->dim, 4 * a->dim};
    const size_t need = a->dw ? (size_t)norm_bwd_slots(a->rows, a->dim) * (size_t)a->dim * 4 : 0;
    if (need) {
        if (!aligned_to(workspace, 16)) return SHAMPOO_E_ARG;
        if (!workspace || bytes < need) return SHAMPOO_E_STATE;
        out[no++] = Area{addr(workspace), 1, (int64_t)need, (int64_t)need};
    }
    if (any_overlap(out, no, in, ni)) return SHAMPOO_E_ARG;
    for (int i = 0; i < no; ++i)
        if (overlap(out[i], dz)) return SHAMPOO_E_ARG;
    NormBwdArgs k{};
    k.g = Wide{addr(a->grad), a->grad_pitch};
    k.z = Wide{addr(a->z), a->z_pitch};
    k.add = Wide{addr(a->add), a->add_pitch};
    k.dz = Wide{addr(a->dz), a->dz_pitch};
    k.w = a->weight;
    k.rstd = a->rstd;
    k.dw = a->dw;
    k.partials = static_cast<float*>(workspace);
    k.rows = a->rows;
    k.dim = a->dim;
    k.w_type = a->weight_type;
    k.accumulate = a->accumulate;
    k.slots = norm_bwd_slots(a->rows, a->dim);
    return status_of(launch_norm_bwd(a->grad_type, a->z_type, k, static_cast<hipStream_t>(stream)));
}

int shampoo_matmul8_workspace(int64_t m, int64_t n, int64_t k, int32_t type, size_t* bytes) {
    if (!bytes || !size_ok(m) || !size_ok(n) || !size_ok(k) || !type_ok(type)) return SHAMPOO_E_ARG;
    *bytes = mul8_workspace(plan_mul8(m, n, k, type), m, n);
    return SHAMPOO_OK;
}

int shampoo_matmul8(const shampoo_matrix8* a, const shampoo_matrix8* b, void* c, int32_t type, int64_t pitch,
                    int32_t accumulate, void* workspace, size_t bytes, void* stream) {
    if (!a || !b || accumulate < 0 || accumulate > 1 || a->cols != b->cols) return SHAMPOO_E_ARG;
    if (!size_ok(a->rows) || !size_ok(b->rows) || !size_ok(a->cols)) return SHAMPOO_E_ARG;
    const int64_t m = a->rows, n = b->rows, k = a->cols;
    Area in[4], out[2];
    int no = 1;
    if (!matrix8(a, m, k, in[0], in[1]) || !matrix8(b, n, k, in[2], in[3])) return SHAMPOO_E_ARG;
    if (!wide(c, type, pitch, m, n, out[0])) return SHAMPOO_E_ARG;
    if (out[0].empty()) return SHAMPOO_OK;
    if (!rows_fit(a) || !rows_fit(b)) return SHAMPOO_E_UNSUPPORTED;
    const Mul8Plan p = plan_mul8(m, n, k, type);
    if (!mul8_fits(p, m, n)) return SHAMPOO_E_UNSUPPORTED;
    const size_t need = mul8_workspace(p, m, n);
    if (need) {
        if (!aligned_to(workspace, 16)) return SHAMPOO_E_ARG;
        if (!workspace || bytes < need) return SHAMPOO_E_STATE;
        out[no++] = Area{addr(workspace), 1, (int64_t)need, (int64_t)need};
    }
    if (any_overlap(out, no, in, 4)) return SHAMPOO_E_ARG;
    Mul8Args g{};
    g.a = device_view(a);
    g.b = device_view(b);
    g.c = Wide{addr(c), pitch};
    g.partials = static_cast<float*>(workspace);
    g.m = m;
    g.n = n;
    g.k = k;
    g.c_type = type;
    g.accumulate = accumulate;
    g.fa = a->format;
    g.fb = b->format;
    g.splits = p.splits;
    g.blocks_per_split = p.blocks_per_split;
    return status_of(launch_mul8(p, g, static_cast<hipStream_t>(stream)));
}

int shampoo_weights8_create(int32_t n, const shampoo_weight_desc* weights, shampoo_weights8_t** out) {
    if (!out) return SHAMPOO_E_ARG;
    *out = nullptr;
    if (!weights || n < 1) return SHAMPOO_E_ARG;
    double tiles = 0;
    for (int i = 0; i < n; ++i) {
        const auto& d = weights[i];
        if (!size_ok(d.rows) || !size_ok(d.cols) || !type_ok(d.type) || d.type != weights[0].type || d.reserved) return SHAMPOO_E_ARG;
        if (d.rows >= (int64_t)1 << 31 || d.cols >= (int64_t)1 << 31) return SHAMPOO_E_UNSUPPORTED;
        tiles += (double)blocks_of(d.rows) * (double)blocks_of(d.cols);
    }
    if (tiles >= (double)kMaxTiles8) return SHAMPOO_E_UNSUPPORTED;
    shampoo_weights8_s* h = nullptr;
    try {
        h = new shampoo_weights8_s;
        h->desc.assign(weights, weights + n);
        h->type = weights[0].type;
        h->tiles.reserve((size_t)tiles);
        int64_t codes = 0, scales = 0;
        for (int i = 0; i < n; ++i) {
            const auto& d = h->desc[i];
            QuantJob j{};
            j.nrows = d.rows;
            j.ncols = d.cols;
            j.x.pitch = d.cols;
            j.rows = placed(d.rows, d.cols, codes, scales);
            j.cols = placed(d.cols, d.rows, codes, scales);
            h->jobs.push_back(j);
            for (int64_t r = 0; r < blocks_of(d.rows); ++r)
                for (int64_t c = 0; c < blocks_of(d.cols); ++c) h->tiles.push_back(QuantTile{i, 0, (int32_t)r, (int32_t)c});
        }
        h->lay.off_codes = 0;
        h->lay.code_bytes = codes;
        h->lay.off_scales = codes;
        h->lay.scale_bytes = scales;
        h->off_jobs = codes + scales;
        h->off_tiles = h->off_jobs + up((int64_t)(h->jobs.size() * sizeof(QuantJob)), 256);
        h->lay.total = up(h->off_tiles + (int64_t)(h->tiles.size() * sizeof(QuantTile)), 256);
    } catch (const std::bad_alloc&) {
        delete h;
        return SHAMPOO_E_NOMEM;
    }
    *out = h;
    return SHAMPOO_OK;
}

int shampoo_weights8_get_layout(const shampoo_weights8_t* h, shampoo_weights8_layout* out) {
    if (!h || !out) return SHAMPOO_E_ARG;
    *out = h->lay;
    return SHAMPOO_OK;
}

int shampoo_weights8_bind_state(shampoo_weights8_t* h, void* dev_state, size_t bytes, void* stream) {
    if (!h || !dev_state || !aligned_to(dev_state, 256)) return SHAMPOO_E_ARG;
    if (bytes < (size_t)h->lay.total) return SHAMPOO_E_STATE;
    hipStream_t s = static_cast<hipStream_t>(stream);
    int device = -1;
    if (hipGetDevice(&device) != hipSuccess) return SHAMPOO_E_HIP;
    std::vector<QuantJob> jobs;
    try {
        jobs = h->jobs;
    } catch (const std::bad_alloc&) {
        return SHAMPOO_E_NOMEM;
    }
    unsigned char* arena = static_cast<unsigned char*>(dev_state);
    for (QuantJob& j : jobs)
        for (Mat8* m : {&j.rows, &j.cols}) {
            m->codes += addr(arena) + (uint64_t)h->lay.off_codes;
            m->scales += addr(arena) + (uint64_t)h->lay.off_scales;
        }
    h->bound = h->weights_bound = false;
    int rc = status_of(hipMemsetAsync(arena, 0, (size_t)h->lay.total, s));
    if (!rc) rc = status_of(hipMemcpyAsync(arena + h->off_jobs, jobs.data(), jobs.size() * sizeof(QuantJob), hipMemcpyHostToDevice, s));
    if (!rc && !h->tiles.empty())
        rc = status_of(hipMemcpyAsync(arena + h->off_tiles, h->tiles.data(), h->tiles.size() * sizeof(QuantTile), hipMemcpyHostToDevice, s));
    const int waited = status_of(hipStreamSynchronize(s));   // before `jobs` goes
    if (rc || waited) return rc ? rc : waited;
    h->arena = arena;
    h->device = device;
    h->bound = true;
    return SHAMPOO_OK;
}

int shampoo_weights8_bind_weights(shampoo_weights8_t* h, const void* const* weights, void* stream) {
    if (!h || !weights) return SHAMPOO_E_ARG;
    if (!h->bound || !on_device(h->device)) return SHAMPOO_E_STATE;
    const int n = (int)h->desc.size();
    const Area state{addr(h->arena), 1, h->lay.total, h->lay.total};
    for (int i = 0; i < n; ++i) {
        const auto& d = h->desc[i];
        Area w;
        if (!wide(weights[i], d.type, d.rows * d.cols, 1, d.rows * d.cols, w) || overlap(w, state)) return SHAMPOO_E_ARG;
    }
    for (int i = 0; i < n; i += kWeightBatch) {
        AddrBatch b{};
        const int m = n - i < kWeightBatch ? n - i : kWeightBatch;
        for (int k = 0; k < m; ++k) b.a[k] = addr(weights[i + k]);
        const int rc = status_of(launch_weights8_bind(reinterpret_cast<QuantJob*>(h->arena + h->off_jobs), i, m, b,
                                                      static_cast<hipStream_t>(stream)));
        if (rc) return rc;
    }
    h->weights_bound = true;
    return SHAMPOO_OK;
}

int shampoo_weights8_refresh(shampoo_weights8_t* h, void* stream) {
    if (!h) return SHAMPOO_E_ARG;
    if (!h->bound || !h->weights_bound || !on_device(h->device)) return SHAMPOO_E_STATE;
    if (h->tiles.empty()) return SHAMPOO_OK;
    return status_of(launch_weights8(h->type, reinterpret_cast<const QuantJob*>(h->arena + h->off_jobs),
                                     reinterpret_cast<const QuantTile*>(h->arena + h->off_tiles), (int)h->tiles.size(),
                                     static_cast<hipStream_t>(stream)));
}

int shampoo_weights8_matrix(const shampoo_weights8_t* h, int32_t i, int32_t transposed, shampoo_matrix8* out) {
    if (!h || !out || i < 0 || i >= (int32_t)h->desc.size() || transposed < 0 || transposed > 1) return SHAMPOO_E_ARG;
    if (!h->bound) return SHAMPOO_E_STATE;
    const QuantJob& j = h->jobs[i];
    const Mat8& m = transposed ? j.cols : j.rows;
    *out = shampoo_matrix8{h->arena + h->lay.off_codes + m.codes, h->arena + h->lay.off_scales + m.scales,
                           transposed ? j.ncols : j.nrows, transposed ? j.nrows : j.ncols, m.pitch, m.spitch, SHAMPOO_E4M3, 0};
    return SHAMPOO_OK;
}

void shampoo_weights8_destroy(shampoo_weights8_t* h) { delete h; }

}  // extern "C"
