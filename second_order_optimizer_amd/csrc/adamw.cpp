// C-ABI of the first-order operators: the plan and launch sequence of one
// AdamW step over many tensors, and of the global gradient norm.
//
// A plan cuts every tensor into runs of 256 elements and hands a few runs to
// each workgroup, so that hundreds of small tensors and a few huge ones are
// one launch.  Nothing is uploaded by a step: the tables lie in the caller's
// state buffer, tensor addresses reach it as kernel arguments when they are
// bound, and the step counter lives on the device, so a step can be captured
// into a graph and replayed.
#include "../../include/shampoo.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstring>
#include <new>
#include <vector>

#include "adamw.hpp"

using namespace shampoo;

namespace {

constexpr int64_t kMaxNumel = (int64_t)1 << 36;
// A step or a norm over more than this passes the caches by: its data would
// not be there at the next step, and what they hold of the program's stays.
// Three plans in turn of 16M fp32 elements: 78 us, 90 through the caches; of
// 4M: 21 us, 19 through them; the norm of 302M bf16 elements: 92 us, 103
// through them.  Of the 256 MiB last-level cache a program leaves a step part.
// What reads the gradients after their norm gains or loses by it (norm and what
// follows, through the caches / past them): clip_into of 120 and 250 MB of fp32
// 70 / 67 and 143 / 131 us; a step of bf16 weights with 8-bit moments 161 / 159
// and 336 / 332; one with fp32 moments, fp32 gradients 148 / 161 and 308 / 336,
// bf16 ones 266 / 283 and 555 / 592.  A norm's plan does not know what follows.
constexpr int64_t kCacheBytes = (int64_t)96 << 20;
constexpr double kMinEps = 0x1p-100;               // sqrt(v) c + eps is a normal number
constexpr int64_t kMaxTiles = ((int64_t)1 << 24) - 1;   // workgroups of 256 threads in a launch
constexpr int64_t kMaxPieces = (int64_t)1 << 26;         // pieces of a norm plan, likewise

int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
int64_t runs_of(int64_t numel) { return (numel + kRun - 1) / kRun; }
int status_of(hipError_t e) { return e == hipSuccess ? SHAMPOO_OK : SHAMPOO_E_HIP; }

size_t dtype_bytes(int dt) { return dt == SHAMPOO_F32 ? 4 : 2; }

bool on_device(int device) {
    int d = -1;
    return hipGetDevice(&d) == hipSuccess && d == device;
}

// Whether any two of these address ranges share a byte.
struct Span {
    uint64_t begin, end;
};
bool overlap(std::vector<Span>& v) {
    std::sort(v.begin(), v.end(), [](const Span& a, const Span& b) { return a.begin < b.begin; });
    for (size_t i = 1; i < v.size(); ++i)
        if (v[i].begin < v[i - 1].end) return true;
    return false;
}
void add_span(std::vector<Span>& v, const void* p, int64_t bytes) {
    if (p && bytes > 0) v.push_back({reinterpret_cast<uint64_t>(p), reinterpret_cast<uint64_t>(p) + (uint64_t)bytes});
}

// The launch of the tensors that share one kernel.
struct Group {
    int param = 0, grad = 0;
    bool bits8 = false;
    std::vector<AdamwTile> tiles;
    int64_t off_tiles = 0, off_clocks = 0;
};

// The step counters of a tensor's workgroups.
struct Clocks {
    int first = 0, n = 0;
};

}  // namespace

struct shampoo_adamw_s {
    shampoo_adamw_config cfg{};
    std::vector<shampoo_adamw_tensor> desc;
    std::vector<AdamwTensor> table;
    std::vector<Group> groups;
    std::vector<Clocks> clocks;   // of each tensor
    bool per_tensor = false;
    shampoo_adamw_layout lay{};
    int64_t off_table = 0;
    int nclocks = 0;
    int64_t step_bytes = 0;   // weights, gradients and moments
    unsigned char* arena = nullptr;
    bool bound = false, params_bound = false, grads_bound = false;
    int device = -1;
};

struct shampoo_gradnorm_s {
    std::vector<NormTensor> table;
    std::vector<NormTile> tiles;
    int pieces = 1;           // pieces of a tile
    int64_t grad_bytes = 0;
    int64_t off_table = 0, off_tiles = 0, off_partials = 0, off_tickets = 0, off_record = 0;
    size_t total = 0;
    unsigned char* arena = nullptr;
    bool bound = false, grads_bound = false, outs_bound = false, computed = false;
    int device = -1;
};

namespace {

AdamwClock clock_at(const shampoo_adamw_config& c, int64_t t) {
    AdamwClock k{};
    k.t = k.k = t;
    k.b1k = std::pow(c.beta1, (double)(t + 1));
    k.b2k = std::pow(c.beta2, (double)(t + 1));
    k.inv1 = 1.0 / (1.0 - k.b1k);
    k.inv_root2 = (float)(1.0 / std::sqrt(1.0 - k.b2k));
    return k;
}

void plan_adamw(shampoo_adamw_s* h) {
    int64_t runs[2] = {0, 0}, rem_runs = 0;
    for (size_t i = 0; i < h->desc.size(); ++i) {
        const auto& d = h->desc[i];
        AdamwTensor t{};
        t.numel = d.numel;
        t.lr_scale = d.lr_scale;
        t.weight_decay = d.weight_decay;
        t.id = (int32_t)i;
        h->step_bytes += d.numel * (int64_t)(4 + dtype_bytes(d.grad_type) + (d.state_bits == 8 ? 2 : 8));
        const int64_t n = runs_of(d.numel);
        int64_t& r = runs[d.state_bits == 8];
        t.state_run = r;
        r += n;
        t.rem_run = rem_runs;
        if (d.param_type == SHAMPOO_BF16) rem_runs += n;
        h->table.push_back(t);
        if (n == 0) continue;
        Group* g = nullptr;
        for (auto& x : h->groups)
            if (x.param == d.param_type && x.grad == d.grad_type && x.bits8 == (d.state_bits == 8)) g = &x;
        if (!g) {
            h->groups.emplace_back();
            g = &h->groups.back();
            g->param = d.param_type;
            g->grad = d.grad_type;
            g->bits8 = d.state_bits == 8;
        }
        for (int64_t k = 0; k < n; k += kTileRuns) g->tiles.push_back({(int32_t)i, 0, k});
    }
    if (h->groups.empty()) {   // nothing but empty tensors: a workgroup that counts steps
        h->groups.emplace_back();
        h->groups[0].tiles.push_back({0, 0, 0});
    }
    int64_t at = 0;
    const auto take = [&at](int64_t bytes) {
        const int64_t o = at;
        at = round_up(at + bytes, 256);
        return o;
    };
    h->clocks.resize(h->desc.size());
    for (auto& g : h->groups) {
        g.off_clocks = (int64_t)h->nclocks * (int64_t)sizeof(AdamwClock);
        for (const auto& t : g.tiles) {   // those of one tensor follow one another
            Clocks& c = h->clocks[t.tensor];
            if (c.n++ == 0) c.first = h->nclocks;
            ++h->nclocks;
        }
    }
    h->lay.off_clock = take((int64_t)h->nclocks * (int64_t)sizeof(AdamwClock));
    h->off_table = take((int64_t)(h->table.size() * sizeof(AdamwTensor)));
    for (auto& g : h->groups) g.off_tiles = take((int64_t)(g.tiles.size() * sizeof(AdamwTile)));
    h->lay.runs32 = runs[0];
    h->lay.runs8 = runs[1];
    h->lay.runs_rem = rem_runs;
    h->lay.off_rem = take(rem_runs * kRun * 2);
    h->lay.off_m = take(runs[0] * kRun * 4);
    h->lay.off_v = take(runs[0] * kRun * 4);
    h->lay.off_m8 = take(runs[1] * kRun);
    h->lay.off_s8 = take(runs[1] * kRun);
    h->lay.off_m_scale = take(runs[1] * 4);
    h->lay.off_s_scale = take(runs[1] * 4);
    h->lay.total = at;
}

AdamwClock* clocks_of(shampoo_adamw_s* h) {
    return reinterpret_cast<AdamwClock*>(h->arena + h->lay.off_clock);
}

int fill_clocks(shampoo_adamw_s* h, int64_t t, hipStream_t s) {
    return status_of(launch_adamw_clock(clocks_of(h), h->nclocks, clock_at(h->cfg, t), 1 | 2, s));
}

bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

NormArgs norm_args(shampoo_gradnorm_s* h) {
    NormArgs a{};
    a.tensors = reinterpret_cast<const NormTensor*>(h->arena + h->off_table);
    a.tiles = reinterpret_cast<const NormTile*>(h->arena + h->off_tiles);
    a.ntiles = (int32_t)h->tiles.size();
    a.pieces = h->pieces;
    a.partials = reinterpret_cast<double*>(h->arena + h->off_partials);
    a.tickets = reinterpret_cast<int32_t*>(h->arena + h->off_tickets);
    a.record = reinterpret_cast<ClipRecord*>(h->arena + h->off_record);
    return a;
}

}  // namespace

extern "C" {

int shampoo_adamw_create(const shampoo_adamw_config* cfg, int32_t n_tensors,
                         const shampoo_adamw_tensor* tensors, shampoo_adamw_t** out) {
    if (!cfg || !tensors || !out || n_tensors < 1) return SHAMPOO_E_ARG;
    *out = nullptr;
    if (!(cfg->beta1 >= 0.0 && cfg->beta1 < 1.0) || !(cfg->beta2 >= 0.0 && cfg->beta2 < 1.0) ||
        !(cfg->eps >= kMinEps && cfg->eps <= 1e30) || cfg->reserved != 0)
        return SHAMPOO_E_ARG;
    int64_t tiles = 0;
    for (int i = 0; i < n_tensors; ++i) {
        const shampoo_adamw_tensor& d = tensors[i];
        if (d.numel < 0 || d.reserved != 0 || !std::isfinite(d.lr_scale) ||
            !std::isfinite(d.weight_decay) || d.weight_decay < 0.0 || d.lr_scale < 0.0)
            return SHAMPOO_E_ARG;
        if (d.param_type < SHAMPOO_F32 || d.param_type > SHAMPOO_F16 || d.grad_type < SHAMPOO_F32 ||
            d.grad_type > SHAMPOO_F16 || (d.state_bits != 8 && d.state_bits != 32))
            return SHAMPOO_E_ARG;
        if (d.param_type == SHAMPOO_F16 || d.numel > kMaxNumel) return SHAMPOO_E_UNSUPPORTED;
        tiles += runs_of(d.numel) / kTileRuns + 1;
        if (tiles > kMaxTiles) return SHAMPOO_E_UNSUPPORTED;
    }
    shampoo_adamw_s* h = new (std::nothrow) shampoo_adamw_s();
    if (!h) return SHAMPOO_E_NOMEM;
    try {
        h->cfg = *cfg;
        h->desc.assign(tensors, tensors + n_tensors);
        plan_adamw(h);
    } catch (const std::bad_alloc&) {
        delete h;
        return SHAMPOO_E_NOMEM;
    }
    *out = h;
    return SHAMPOO_OK;
}

int shampoo_adamw_get_layout(const shampoo_adamw_t* h, shampoo_adamw_layout* out) {
    if (!h || !out) return SHAMPOO_E_ARG;
    *out = h->lay;
    return SHAMPOO_OK;
}

int shampoo_adamw_tensor_runs(const shampoo_adamw_t* h, int32_t tensor, int64_t* state_run,
                              int64_t* rem_run) {
    if (!h || tensor < 0 || tensor >= (int32_t)h->table.size()) return SHAMPOO_E_ARG;
    const bool rem = h->desc[tensor].param_type == SHAMPOO_BF16;
    if (state_run) *state_run = h->table[tensor].state_run;
    if (rem_run) *rem_run = rem ? h->table[tensor].rem_run : -1;
    return SHAMPOO_OK;
}

int shampoo_adamw_set_counting(shampoo_adamw_t* h, int32_t per_tensor) {
    if (!h || (per_tensor != 0 && per_tensor != 1)) return SHAMPOO_E_ARG;
    if (h->bound) return SHAMPOO_E_STATE;
    h->per_tensor = per_tensor == 1;
    return SHAMPOO_OK;
}

int shampoo_adamw_tensor_count(const shampoo_adamw_t* h, int32_t tensor, int64_t* offset) {
    if (!h || !offset || tensor < 0 || tensor >= (int32_t)h->table.size()) return SHAMPOO_E_ARG;
    const Clocks& c = h->clocks[tensor];
    *offset = c.n ? h->lay.off_clock + (int64_t)c.first * (int64_t)sizeof(AdamwClock) +
                        (int64_t)offsetof(AdamwClock, k)
                  : -1;
    return SHAMPOO_OK;
}

int shampoo_adamw_bind_state(shampoo_adamw_t* h, void* dev_state, size_t bytes, void* stream) {
    if (!h || !dev_state || !aligned_to(dev_state, 256)) return SHAMPOO_E_ARG;
    if (bytes < (size_t)h->lay.total) return SHAMPOO_E_STATE;
    hipStream_t s = static_cast<hipStream_t>(stream);
    h->bound = h->params_bound = h->grads_bound = false;
    if (hipGetDevice(&h->device) != hipSuccess) return SHAMPOO_E_HIP;
    h->arena = static_cast<unsigned char*>(dev_state);
    int rc = status_of(hipMemsetAsync(h->arena, 0, (size_t)h->lay.total, s));
    if (rc) return rc;
    rc = status_of(hipMemcpyAsync(h->arena + h->off_table, h->table.data(),
                                  h->table.size() * sizeof(AdamwTensor), hipMemcpyHostToDevice, s));
    if (rc) return rc;
    for (const auto& g : h->groups) {
        rc = status_of(hipMemcpyAsync(h->arena + g.off_tiles, g.tiles.data(),
                                      g.tiles.size() * sizeof(AdamwTile), hipMemcpyHostToDevice, s));
        if (rc) return rc;
    }
    rc = fill_clocks(h, 0, s);
    if (rc) return rc;
    rc = status_of(hipStreamSynchronize(s));
    if (rc) return rc;
    h->bound = true;
    return SHAMPOO_OK;
}

int shampoo_adamw_bind_tensors(shampoo_adamw_t* h, void* const* params, const void* const* grads,
                               void* stream) {
    if (!h || (!params && !grads)) return SHAMPOO_E_ARG;
    if (!h->bound || !on_device(h->device)) return SHAMPOO_E_STATE;
    const int n = (int)h->desc.size();
    for (int i = 0; i < n; ++i) {
        const shampoo_adamw_tensor& d = h->desc[i];
        if (d.numel == 0) continue;
        if (params && (!params[i] || !aligned_to(params[i], dtype_bytes(d.param_type))))
            return SHAMPOO_E_ARG;
        if (grads && !aligned_to(grads[i], dtype_bytes(d.grad_type))) return SHAMPOO_E_ARG;
    }
    if (params) {   // a weight that is listed twice would be updated by two waves at once
        try {
            std::vector<Span> spans;
            for (int i = 0; i < n; ++i)
                add_span(spans, params[i], h->desc[i].numel * (int64_t)dtype_bytes(h->desc[i].param_type));
            if (overlap(spans)) return SHAMPOO_E_ARG;
        } catch (const std::bad_alloc&) {
            return SHAMPOO_E_NOMEM;
        }
    }
    AdamwTensor* table = reinterpret_cast<AdamwTensor*>(h->arena + h->off_table);
    for (int i = 0; i < n; i += kBindBatch) {
        PtrBatch b{};
        const int m = std::min(kBindBatch, n - i);
        for (int k = 0; k < m; ++k) {
            b.a[k] = params ? reinterpret_cast<uint64_t>(params[i + k]) : 0;
            b.b[k] = grads ? reinterpret_cast<uint64_t>(grads[i + k]) : 0;
        }
        const int rc = status_of(launch_adamw_bind(table, i, m, b, (params ? 1 : 0) | (grads ? 2 : 0),
                                                   static_cast<hipStream_t>(stream)));
        if (rc) return rc;
    }
    h->params_bound |= params != nullptr;
    h->grads_bound |= grads != nullptr;
    return SHAMPOO_OK;
}

int shampoo_adamw_set_step(shampoo_adamw_t* h, int64_t t, void* stream) {
    if (!h || t < 0) return SHAMPOO_E_ARG;
    if (!h->bound || !on_device(h->device)) return SHAMPOO_E_STATE;
    return fill_clocks(h, t, static_cast<hipStream_t>(stream));
}

int shampoo_adamw_set_tensor_steps(shampoo_adamw_t* h, const int64_t* steps, void* stream) {
    if (!h || !steps) return SHAMPOO_E_ARG;
    if (!h->per_tensor || !h->bound || !on_device(h->device)) return SHAMPOO_E_STATE;
    for (size_t i = 0; i < h->desc.size(); ++i)
        if (steps[i] < 0) return SHAMPOO_E_ARG;
    for (size_t i = 0; i < h->desc.size(); ++i) {
        const Clocks& c = h->clocks[i];
        if (!c.n) continue;
        const int rc = status_of(launch_adamw_clock(clocks_of(h) + c.first, c.n, clock_at(h->cfg, steps[i]), 2,
                                                    static_cast<hipStream_t>(stream)));
        if (rc) return rc;
    }
    return SHAMPOO_OK;
}

int shampoo_adamw_step(shampoo_adamw_t* h, double lr, const float* dev_lr,
                       const shampoo_clip_record* dev_clip, void* stream) {
    if (!h || !std::isfinite(lr) || !aligned_to(dev_lr, 4) || !aligned_to(dev_clip, 16))
        return SHAMPOO_E_ARG;
    if (!h->bound || !h->params_bound || !h->grads_bound || !on_device(h->device))
        return SHAMPOO_E_STATE;
    static_assert(sizeof(shampoo_clip_record) == sizeof(ClipRecord), "record layout");
    const shampoo_adamw_config& c = h->cfg;
    AdamwArgs a{};
    a.tensors = reinterpret_cast<const AdamwTensor*>(h->arena + h->off_table);
    a.clip = reinterpret_cast<const ClipRecord*>(dev_clip);
    a.lr_dev = dev_lr;
    a.lr = lr;
    a.beta1 = c.beta1;
    a.beta2 = c.beta2;
    a.b1 = (float)c.beta1;
    a.c1 = (float)(1.0 - c.beta1);
    a.b2 = (float)c.beta2;
    a.c2 = (float)(1.0 - c.beta2);
    a.eps = (float)c.eps;
    a.seed_mixed = mix32(c.seed);
    a.m = reinterpret_cast<float*>(h->arena + h->lay.off_m);
    a.v = reinterpret_cast<float*>(h->arena + h->lay.off_v);
    a.m8 = h->arena + h->lay.off_m8;
    a.s8 = h->arena + h->lay.off_s8;
    a.m_scale = reinterpret_cast<float*>(h->arena + h->lay.off_m_scale);
    a.s_scale = reinterpret_cast<float*>(h->arena + h->lay.off_s_scale);
    a.rem = reinterpret_cast<int16_t*>(h->arena + h->lay.off_rem);
    a.stream_past = h->step_bytes > kCacheBytes;
    a.per_tensor = h->per_tensor;
    for (const auto& g : h->groups) {
        a.tiles = reinterpret_cast<const AdamwTile*>(h->arena + g.off_tiles);
        a.ntiles = (int32_t)g.tiles.size();
        a.clocks = reinterpret_cast<AdamwClock*>(h->arena + h->lay.off_clock + g.off_clocks);
        const int rc = status_of(launch_adamw(g.param, g.grad, g.bits8, a, static_cast<hipStream_t>(stream)));
        if (rc) return rc;
    }
    return SHAMPOO_OK;
}

void shampoo_adamw_destroy(shampoo_adamw_t* h) { delete h; }

int shampoo_gradnorm_create(int32_t n_tensors, const shampoo_grad_desc* tensors,
                            shampoo_gradnorm_t** out) {
    if (!tensors || !out || n_tensors < 1) return SHAMPOO_E_ARG;
    *out = nullptr;
    int64_t tiles = 0;
    for (int i = 0; i < n_tensors; ++i) {
        const shampoo_grad_desc& d = tensors[i];
        if (d.numel < 0 || d.reserved != 0 || d.dtype < SHAMPOO_F32 || d.dtype > SHAMPOO_F16)
            return SHAMPOO_E_ARG;
        if (d.numel > kMaxNumel) return SHAMPOO_E_UNSUPPORTED;
        tiles += d.numel / kNormPiece + 1;
        if (tiles > kMaxPieces) return SHAMPOO_E_UNSUPPORTED;
    }
    shampoo_gradnorm_s* h = new (std::nothrow) shampoo_gradnorm_s();
    if (!h) return SHAMPOO_E_NOMEM;
    // twice the work for one reading of the tables once every wave has several
    // (302M bf16 elements: 92 us, 93 with one piece, 99 with four)
    h->pieces = tiles >= 8 * 8192 ? 2 : 1;
    try {
        const int64_t per_tile = (int64_t)h->pieces * kNormPiece;
        for (int i = 0; i < n_tensors; ++i) {
            NormTensor t{};
            t.numel = tensors[i].numel;
            t.dtype = tensors[i].dtype;
            h->table.push_back(t);
            h->grad_bytes += t.numel * (int64_t)dtype_bytes(t.dtype);
            for (int64_t k = 0; k < t.numel; k += per_tile) h->tiles.push_back({i, 0, k});
        }
    } catch (const std::bad_alloc&) {
        delete h;
        return SHAMPOO_E_NOMEM;
    }
    int64_t at = 0;
    const auto take = [&at](int64_t bytes) {
        const int64_t o = at;
        at = round_up(at + bytes, 256);
        return o;
    };
    h->off_record = take(sizeof(ClipRecord));
    h->off_tickets = take(128 * (kNormGroups + 1));
    h->off_partials = take(8 * (int64_t)norm_grid((int64_t)h->tiles.size()));
    h->off_table = take((int64_t)(h->table.size() * sizeof(NormTensor)));
    h->off_tiles = take((int64_t)(h->tiles.size() * sizeof(NormTile)));
    h->total = (size_t)at;
    *out = h;
    return SHAMPOO_OK;
}

int shampoo_gradnorm_state_bytes(const shampoo_gradnorm_t* h, size_t* bytes) {
    if (!h || !bytes) return SHAMPOO_E_ARG;
    *bytes = h->total;
    return SHAMPOO_OK;
}

int shampoo_gradnorm_bind_state(shampoo_gradnorm_t* h, void* dev_state, size_t bytes, void* stream) {
    if (!h || !dev_state || !aligned_to(dev_state, 256)) return SHAMPOO_E_ARG;
    if (bytes < h->total) return SHAMPOO_E_STATE;
    hipStream_t s = static_cast<hipStream_t>(stream);
    h->bound = h->grads_bound = h->outs_bound = h->computed = false;
    if (hipGetDevice(&h->device) != hipSuccess) return SHAMPOO_E_HIP;
    h->arena = static_cast<unsigned char*>(dev_state);
    int rc = status_of(hipMemsetAsync(h->arena, 0, h->total, s));
    if (rc) return rc;
    rc = status_of(hipMemcpyAsync(h->arena + h->off_table, h->table.data(),
                                  h->table.size() * sizeof(NormTensor), hipMemcpyHostToDevice, s));
    if (rc) return rc;
    if (!h->tiles.empty()) {
        rc = status_of(hipMemcpyAsync(h->arena + h->off_tiles, h->tiles.data(),
                                      h->tiles.size() * sizeof(NormTile), hipMemcpyHostToDevice, s));
        if (rc) return rc;
    }
    // no norm yet (a captured one only runs with its graph): a step that reads
    // the record changes nothing
    const ClipRecord none{0.f, 0.f, 1, 0};
    rc = status_of(hipMemcpyAsync(h->arena + h->off_record, &none, sizeof none, hipMemcpyHostToDevice, s));
    if (rc) return rc;
    rc = status_of(hipStreamSynchronize(s));
    if (rc) return rc;
    h->bound = true;
    return SHAMPOO_OK;
}

int shampoo_gradnorm_bind_grads(shampoo_gradnorm_t* h, const void* const* grads, float* const* outs,
                                void* stream) {
    if (!h || !grads) return SHAMPOO_E_ARG;
    if (!h->bound || !on_device(h->device)) return SHAMPOO_E_STATE;
    const int n = (int)h->table.size();
    for (int i = 0; i < n; ++i) {
        const NormTensor& t = h->table[i];
        if (t.numel == 0) continue;
        if (!aligned_to(grads[i], dtype_bytes(t.dtype))) return SHAMPOO_E_ARG;
        if (outs && !aligned_to(outs[i], 4)) return SHAMPOO_E_ARG;
    }
    if (outs) {
        // outputs overlap neither each other nor a gradient, but for an fp32
        // gradient that is its own output
        try {
            std::vector<Span> spans;
            for (int i = 0; i < n; ++i) {
                const NormTensor& t = h->table[i];
                add_span(spans, outs[i], 4 * t.numel);
            }
            if (overlap(spans)) return SHAMPOO_E_ARG;
            for (int i = 0; i < n; ++i) {
                const NormTensor& t = h->table[i];
                if (outs[i] && (const void*)outs[i] == grads[i] && t.dtype == SHAMPOO_F32) continue;
                const uint64_t b = reinterpret_cast<uint64_t>(grads[i]);
                const uint64_t e = b + (uint64_t)t.numel * dtype_bytes(t.dtype);
                if (!b || t.numel == 0) continue;
                // the spans are sorted and apart: the first that ends after b
                const auto it = std::upper_bound(spans.begin(), spans.end(), b,
                                                 [](uint64_t x, const Span& s) { return x < s.end; });
                if (it != spans.end() && it->begin < e) return SHAMPOO_E_ARG;
            }
        } catch (const std::bad_alloc&) {
            return SHAMPOO_E_NOMEM;
        }
    }
    NormTensor* table = reinterpret_cast<NormTensor*>(h->arena + h->off_table);
    for (int i = 0; i < n; i += kBindBatch) {
        PtrBatch b{};
        const int m = std::min(kBindBatch, n - i);
        for (int k = 0; k < m; ++k) {
            b.a[k] = reinterpret_cast<uint64_t>(grads[i + k]);
            b.b[k] = outs ? reinterpret_cast<uint64_t>(outs[i + k]) : 0;
        }
        const int rc = status_of(launch_norm_bind(table, i, m, b, static_cast<hipStream_t>(stream)));
        if (rc) return rc;
    }
    h->grads_bound = true;
    h->outs_bound = outs != nullptr;
    return SHAMPOO_OK;
}

int shampoo_gradnorm_compute(shampoo_gradnorm_t* h, double max_norm, double grad_scale, void* stream) {
    if (!h || !(max_norm > 0.0) || !(grad_scale > 0.0 && std::isfinite(grad_scale)))
        return SHAMPOO_E_ARG;
    if (!h->bound || !h->grads_bound || !on_device(h->device)) return SHAMPOO_E_STATE;
    NormArgs a = norm_args(h);
    a.stream_past = h->grad_bytes > kCacheBytes;
    a.max_norm = max_norm;
    a.grad_scale = grad_scale;
    const int rc = status_of(launch_norm(a, static_cast<hipStream_t>(stream)));
    h->computed |= rc == SHAMPOO_OK;
    return rc;
}

int shampoo_gradnorm_clip_into(shampoo_gradnorm_t* h, void* stream) {
    if (!h) return SHAMPOO_E_ARG;
    if (!h->bound || !h->outs_bound || !h->computed || !on_device(h->device)) return SHAMPOO_E_STATE;
    if (h->tiles.empty()) return SHAMPOO_OK;
    return status_of(launch_clip(norm_args(h), static_cast<hipStream_t>(stream)));
}

int shampoo_gradnorm_record(const shampoo_gradnorm_t* h, const shampoo_clip_record** dev_record) {
    if (!h || !dev_record) return SHAMPOO_E_ARG;
    if (!h->bound) return SHAMPOO_E_STATE;
    *dev_record = reinterpret_cast<const shampoo_clip_record*>(h->arena + h->off_record);
    return SHAMPOO_OK;
}

void shampoo_gradnorm_destroy(shampoo_gradnorm_t* h) { delete h; }

}  // extern "C"
