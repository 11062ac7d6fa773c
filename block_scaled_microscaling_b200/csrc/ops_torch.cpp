// ops_torch.cpp -- the operators' calls with torch tensors, in C++ (module _ops of the package).
//
// ops.py documents the helpers, checks their arguments and calls the C entry points of libmxq through ctypes. For the
// plain case (the library's types, matching shapes, contiguous where that is asked for, default options) the same
// calls are made here, where allocating the outputs, the checks and the autograd node take a few microseconds
// together; a kernel of a small batch takes no more. Anything else returns None (or False), and ops.py goes its own way,
// which raises the errors: no rule is relaxed here. The two training functions exist here alone. Linked against
// libmxq.so beside it.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAStream.h>
#include <pybind11/pybind11.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>

#include "../../include/mxq_ops.h"

namespace {

namespace py = pybind11;
using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;

bool values(const Tensor& t) { return t.is_cuda() && (t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kFloat); }
bool bytes(const Tensor& t) { return t.is_cuda() && t.scalar_type() == at::kByte && t.is_contiguous(); }
mxq_dtype dtype_of(const Tensor& t) { return t.scalar_type() == at::kFloat ? MXQ_F32 : MXQ_BF16; }
mxq_stream stream_of(const Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }
int64_t payload(int fmt) { return fmt == MXQ_MXFP4_E2M1 ? 16 : 32; }
bool product_format(int fmt) { return fmt == MXQ_MXFP4_E2M1 || fmt == MXQ_MXFP8_E4M3; }
// t as the C entry points read it: contiguous, on a 16-byte boundary (a slice, such as a gradient that cat() hands back, may
// begin anywhere)
Tensor dense(const Tensor& t) {
    const Tensor c = t.contiguous();
    return reinterpret_cast<uintptr_t>(c.const_data_ptr()) % 16 == 0 ? c : c.clone();
}
Tensor scratch(int64_t n, const Tensor& like) { return at::empty({n}, like.options().dtype(at::kByte)); }

void ok(mxq_status s, const char* what) {
    TORCH_CHECK(s == MXQ_OK, what, ": status ", static_cast<int>(s), " (", mxq_status_string(s), ")");
}

// ---- linear -------------------------------------------------------------------------------------

std::optional<Tensor> linear(const Tensor& x, const Tensor& w_codes, const Tensor& w_scales, int fmt) {
    if (!product_format(fmt) || !values(x) || x.dim() == 0 || !x.is_contiguous() || !bytes(w_codes) || !bytes(w_scales) ||
        w_codes.dim() != 2)
        return std::nullopt;
    const int64_t k = x.size(-1);
    if (k <= 0 || k % 32 != 0) return std::nullopt;
    const int64_t m = x.numel() / k, n = w_codes.size(0);
    if (w_codes.size(1) != k / 32 * payload(fmt) || (size_t)w_scales.numel() < mxq_mma_scales_bytes(n, k)) return std::nullopt;
    auto shape = x.sizes().vec();
    shape.back() = n;
    at::NoGradGuard no_grad;
    Tensor out = at::empty(shape, x.options());
    const size_t need = mxq_linear_workspace_bytes((mxq_format)fmt, m, k);
    Tensor ws = scratch((int64_t)need, x);
    if (mxq_linear((mxq_format)fmt, x.const_data_ptr(), dtype_of(x), m, k, w_codes.const_data_ptr(), w_scales.const_data_ptr(), n,
                   out.mutable_data_ptr(), ws.mutable_data_ptr(), need, stream_of(x)) != MXQ_OK)
        return std::nullopt;
    return out;
}

// codes and tile-layout scales of a [rows, cols] operand that lie one after the other
struct Operand {
    char *codes = nullptr, *scales = nullptr;
    int64_t end = 0;  // bytes from the allocation's start
};
int64_t operand_bytes(int fmt, int64_t rows, int64_t cols) {
    return rows * (cols / 32) * payload(fmt) + (rows + 127) / 128 * 128 * ((cols + 127) / 128 * 4);
}
Operand operand(const Tensor& buf, int64_t at, int fmt, int64_t rows, int64_t cols) {
    char* const p = static_cast<char*>(buf.mutable_data_ptr()) + at;
    return {p, p + rows * (cols / 32) * payload(fmt), at + operand_bytes(fmt, rows, cols)};
}
void quantize(const Tensor& x, const Operand& row, int row_fmt, const Operand& col, int col_fmt) {
    ok(mxq_quantize_both((mxq_format)row_fmt, (mxq_format)col_fmt, x.const_data_ptr(), dtype_of(x), x.size(0), x.size(1), row.codes,
                         row.scales, col.codes, col.scales, stream_of(x)),
       "mxq_quantize_both");
}
void product(const Operand& a, const Operand& b, int fmt, int64_t m, int64_t n, int64_t k, const Tensor& out) {
    ok(mxq_matmul((mxq_format)fmt, a.codes, a.scales, b.codes, b.scales, m, n, k, out.mutable_data_ptr(), dtype_of(out), stream_of(out)),
       "mxq_matmul");
}

// gradients whose own derivative raises (under create_graph)
variable_list once(variable_list grads) {
    if (!at::GradMode::is_enabled()) return grads;
    variable_list in;
    for (auto& g : grads)
        if (g.defined()) in.push_back(g.detach().requires_grad_(true));
    auto node = std::make_shared<torch::autograd::DelayedError>("the gradients of this operator are not differentiable", (int64_t)in.size());
    variable_list out = (*node)(std::move(in));
    size_t i = 0;
    for (auto& g : grads)
        if (g.defined()) g = out[i++];
    return grads;
}

struct LinearSTE : torch::autograd::Function<LinearSTE> {
    static Tensor forward(AutogradContext* ctx, const Tensor& x, const Tensor& weight, int64_t fmt, bool need_dx, bool need_dw) {
        const int64_t k = weight.size(1), n = weight.size(0), m = x.numel() / k, m32 = (m + 31) / 32 * 32;
        auto shape = x.sizes().vec();
        shape.back() = n;
        Tensor y = at::empty(shape, x.options()), kept;
        // the checkpoint is the operand of the weight's gradient: x rounded along the tokens
        if (need_dw) kept = scratch(operand_bytes(MXQ_MXFP8_E4M3, k, m32), x);
        if (m > 0) {
            const Tensor x2 = dense(x.reshape({m, k})), w = dense(weight);
            Tensor buf = scratch(operand_bytes((int)fmt, m, k) + operand_bytes((int)fmt, n, k), x);
            const Operand a = operand(buf, 0, (int)fmt, m, k), b = operand(buf, a.end, (int)fmt, n, k);
            quantize(x2, a, (int)fmt, need_dw ? operand(kept, 0, MXQ_MXFP8_E4M3, k, m32) : Operand(), MXQ_MXFP8_E4M3);
            quantize(w, b, (int)fmt, Operand(), MXQ_MXFP8_E4M3);
            product(a, b, (int)fmt, m, n, k, y);
        }
        ctx->save_for_backward({need_dx ? weight : Tensor(), kept});
        ctx->saved_data["x"] = x.sizes().vec();
        ctx->saved_data["n"] = n;
        ctx->saved_data["types"] = std::vector<int64_t>{(int64_t)x.scalar_type(), (int64_t)weight.scalar_type()};
        return y;
    }
    static variable_list backward(AutogradContext* ctx, variable_list grads) {
        const auto saved = ctx->get_saved_variables();
        const Tensor &weight = saved[0], &kept = saved[1];
        const auto shape = ctx->saved_data["x"].toIntVector(), types = ctx->saved_data["types"].toIntVector();
        const int64_t k = shape.back(), n = ctx->saved_data["n"].toInt();
        Tensor dx, dw;
        {
            at::NoGradGuard no_grad;
            const int64_t m = grads[0].numel() / n, m32 = (m + 31) / 32 * 32;
            const Tensor g = dense(grads[0].reshape({m, n}));
            constexpr int f = MXQ_MXFP8_E4M3;
            if (m == 0) {  // no tokens
                if (weight.defined()) dx = at::empty(shape, g.options().dtype((at::ScalarType)types[0]));
                if (kept.defined()) dw = at::zeros({n, k}, g.options().dtype((at::ScalarType)types[1]));
                return {dx, dw, Tensor(), Tensor(), Tensor()};
            }
            int64_t need = weight.defined() ? operand_bytes(f, m, n) + operand_bytes(f, k, n) : 0;
            if (kept.defined()) need += operand_bytes(f, n, m32);
            Tensor buf = scratch(need, g);
            Operand row, wt, col;
            if (weight.defined()) {
                row = operand(buf, 0, f, m, n);
                wt = operand(buf, row.end, f, k, n);
            }
            if (kept.defined()) col = operand(buf, wt.end, f, n, m32);
            if (weight.defined() || kept.defined()) quantize(g, row, f, col, f);
            if (weight.defined()) {
                quantize(dense(weight), Operand(), f, wt, f);
                dx = at::empty(shape, g.options().dtype((at::ScalarType)types[0]));
                product(row, wt, f, m, k, n, dx);
            }
            if (kept.defined()) {
                dw = at::empty({n, k}, g.options().dtype((at::ScalarType)types[1]));
                product(col, operand(kept, 0, f, k, m32), f, n, k, m32, dw);
            }
        }
        variable_list out = once({dx, dw});
        return {out[0], out[1], Tensor(), Tensor(), Tensor()};
    }
};

std::optional<Tensor> linear_ste(const Tensor& x, const Tensor& weight, int fmt) {
    if (!product_format(fmt) || !values(x) || !values(weight) || x.dim() == 0 || weight.dim() != 2 ||
        x.size(-1) != weight.size(1) || weight.size(0) <= 0 || weight.size(0) % 32 != 0 || weight.size(1) <= 0 ||
        weight.size(1) % 32 != 0 ||
        x.device() != weight.device())
        return std::nullopt;
    const bool grad = at::GradMode::is_enabled();
    return LinearSTE::apply(x, weight, (int64_t)fmt, grad && x.requires_grad(), grad && weight.requires_grad());
}

// ---- swiglu -------------------------------------------------------------------------------------

// gate's codes and scales and up's in one allocation of 66 bytes per block (codes first: aligned)
struct Checkpoint {
    char *gc = nullptr, *gs = nullptr, *uc = nullptr, *us = nullptr;
    Checkpoint() = default;
    Checkpoint(const Tensor& buf, int64_t n) {
        gc = static_cast<char*>(buf.mutable_data_ptr());
        uc = gc + n;
        gs = gc + 2 * n;
        us = gs + n / 32;
    }
};

// values between rows if the leading dimensions of t are one dimension of rows, which do not overlap (a broadcast
// dimension has the stride 0), whose values are contiguous and whose start and stride are 16-byte aligned; else 0
int64_t row_stride(const Tensor& t) {
    if (t.stride(-1) != 1) return 0;
    int64_t ld = t.size(-1), n = 1;
    bool one = true;  // no dimension of more than one row so far
    for (int64_t i = t.dim() - 2; i >= 0; --i) {
        if (t.size(i) == 1) continue;
        if (one) ld = t.stride(i);
        else if (t.stride(i) != ld * n) return 0;
        one = false;
        n *= t.size(i);
    }
    const bool aligned = ld * t.element_size() % 16 == 0 && reinterpret_cast<uintptr_t>(t.const_data_ptr()) % 16 == 0;
    return ld >= t.size(-1) && aligned ? ld : 0;
}

struct SwiGLU : torch::autograd::Function<SwiGLU> {
    // gate and up, of one shape; or gate alone with up's columns behind its own
    static Tensor forward(AutogradContext* ctx, const Tensor& gate_in, const std::optional<Tensor>& up_in, bool keep) {
        const bool packed = !up_in.has_value();
        Tensor gate = gate_in, up = packed ? Tensor() : *up_in;
        int64_t ld = packed ? 0 : row_stride(gate);
        if (ld == 0 || row_stride(up) != ld) {
            gate = dense(gate);
            if (!packed) up = dense(up);
            ld = gate.size(-1);
        }
        const int64_t cols = gate.size(-1) / (packed ? 2 : 1), rows = gate.numel() / gate.size(-1), n = rows * cols;
        auto shape = gate.sizes().vec();
        shape.back() = cols;
        Tensor out = at::empty(shape, gate.options().memory_format(at::MemoryFormat::Contiguous)), kept;
        Checkpoint c;
        if (keep) {
            kept = scratch(n / 32 * 66, gate);
            c = Checkpoint(kept, n);
        }
        const char* const pg = static_cast<const char*>(gate.const_data_ptr());
        ok(mxq_swiglu_forward(pg, packed ? pg + cols * gate.element_size() : up.const_data_ptr(), dtype_of(gate), rows, cols, ld,
                              out.mutable_data_ptr(), c.gc, c.gs, c.uc, c.us, stream_of(gate)),
           "mxq_swiglu_forward");
        ctx->save_for_backward({kept});
        ctx->saved_data["packed"] = packed;
        return out;
    }
    static variable_list backward(AutogradContext* ctx, variable_list grads) {
        const Tensor kept = ctx->get_saved_variables()[0];
        const bool packed = ctx->saved_data["packed"].toBool();
        Tensor dgate, dup;
        {
            at::NoGradGuard no_grad;
            const Tensor g = dense(grads[0]);
            const int64_t cols = g.size(-1), rows = g.numel() / cols;
            const Checkpoint c(kept, rows * cols);
            char *pg, *pu;
            if (packed) {
                auto shape = g.sizes().vec();
                shape.back() = 2 * cols;
                dgate = at::empty(shape, g.options());
                pg = static_cast<char*>(dgate.mutable_data_ptr());
                pu = pg + cols * g.element_size();
            } else {
                dgate = at::empty_like(g);
                dup = at::empty_like(g);
                pg = static_cast<char*>(dgate.mutable_data_ptr());
                pu = static_cast<char*>(dup.mutable_data_ptr());
            }
            ok(mxq_swiglu_backward(g.const_data_ptr(), dtype_of(g), c.gc, c.gs, c.uc, c.us, rows, cols, pg, pu,
                                   packed ? 2 * cols : cols, stream_of(g)),
               "mxq_swiglu_backward");
        }
        variable_list out = once({dgate, dup});
        return {out[0], out[1], Tensor()};
    }
};

std::optional<Tensor> swiglu(const Tensor& gate, const std::optional<Tensor>& up) {
    if (!values(gate) || gate.dim() == 0 || gate.size(-1) <= 0 || gate.size(-1) % (up ? 32 : 64) != 0) return std::nullopt;
    if (up && (up->sizes() != gate.sizes() || up->scalar_type() != gate.scalar_type() ||
               up->device() != gate.device()))
        return std::nullopt;
    const bool keep = at::GradMode::is_enabled() && (gate.requires_grad() || (up && up->requires_grad()));
    return SwiGLU::apply(gate, up, keep);
}

// ---- the cache ----------------------------------------------------------------------------------

struct Cache {
    Tensor kc, ks, vc, vs;
    mxq_kv_cache c{};
    const mxq_kv_cache* raw() {  // with the pointers of now
        c.k_codes = kc.mutable_data_ptr();
        c.k_scales = ks.mutable_data_ptr();
        c.v_codes = vc.mutable_data_ptr();
        c.v_scales = vs.mutable_data_ptr();
        return &c;
    }
};
std::optional<Cache> cache(const Tensor& kc, const Tensor& ks, const Tensor& vc, const Tensor& vs) {
    for (const Tensor* t : {&kc, &ks, &vc, &vs})
        if (!bytes(*t) || t->dim() != 4) return std::nullopt;
    const auto s = kc.sizes(), e = ks.sizes();
    if (vc.sizes() != s || vs.sizes() != e || e[0] != s[0] || e[1] != s[1] || e[2] != s[2] || e[3] != s[3] / 16 || s[1] < 1 ||
        s[2] < 1 || s[3] < 16 || s[1] > 65536 || s[2] > 65536 || s[3] > 65536)
        return std::nullopt;
    Cache x{kc, ks, vc, vs, {}};
    x.c.pages = s[0];
    x.c.kv_heads = (int32_t)s[1];
    x.c.page_size = (int32_t)s[2];
    x.c.head_dim = (int32_t)(s[3] * 2);
    return x;
}

bool token_rows(const Tensor& t, const Cache& c) {
    return values(t) && t.dim() == 3 && t.size(1) == c.c.kv_heads && t.size(2) == c.c.head_dim && t.stride(2) == 1 &&
           (c.c.kv_heads == 1 || t.stride(1) == c.c.head_dim);
}
bool ints(const Tensor& t, at::ScalarType type) { return t.is_cuda() && t.scalar_type() == type && t.is_contiguous(); }

bool kv_append(Cache& c, const Tensor& k, const Tensor& v, const Tensor& slots) {
    if (!token_rows(k, c) || !token_rows(v, c) || k.size(0) != v.size(0) || k.scalar_type() != v.scalar_type() ||
        !ints(slots, at::kLong) || slots.numel() != k.size(0))
        return false;
    const int64_t n = k.size(0), row = (int64_t)c.c.kv_heads * c.c.head_dim;
    return mxq_kv_append(c.raw(), k.const_data_ptr(), n > 1 ? k.stride(0) : row, v.const_data_ptr(), n > 1 ? v.stride(0) : row, dtype_of(k),
                         n, slots.const_data_ptr<int64_t>(), stream_of(k)) == MXQ_OK;
}

std::optional<std::pair<Tensor, Tensor>> kv_read(Cache& c, const Tensor& slots) {
    if (!ints(slots, at::kLong)) return std::nullopt;
    const auto opts = c.kc.options().dtype(at::kBFloat16);
    Tensor k = at::empty({slots.numel(), c.c.kv_heads, c.c.head_dim}, opts), v = at::empty({slots.numel(), c.c.kv_heads, c.c.head_dim}, opts);
    if (mxq_kv_read(c.raw(), slots.const_data_ptr<int64_t>(), slots.numel(), k.mutable_data_ptr(), v.mutable_data_ptr(), MXQ_BF16,
                    stream_of(slots)) != MXQ_OK)
        return std::nullopt;
    return std::make_pair(k, v);
}

std::optional<Tensor> kv_attention(Cache& c, const Tensor& q, const Tensor& table, const Tensor& lens,
                                   const std::optional<Tensor>& starts, std::optional<int64_t> max_q, std::optional<double> scale,
                                   int64_t window, std::optional<int64_t> max_keys) {
    if (!q.is_cuda() || q.scalar_type() != at::kBFloat16 || q.dim() != 3 || q.size(2) != c.c.head_dim || q.stride(2) != 1 ||
        !ints(lens, at::kInt) || !ints(table, at::kInt) || table.dim() != 2)
        return std::nullopt;
    const int64_t rows = q.size(0), heads = q.size(1), batch = lens.numel();
    if (rows == 0 || heads == 0 || heads % c.c.kv_heads != 0 || heads > 0x7FFFFFFF || batch == 0 || table.size(0) != batch || window < 0 ||
        window > 0x7FFFFFFF || rows > 0x7FFFFFFE)
        return std::nullopt;
    int64_t most_q;
    if (starts) {
        if (!ints(*starts, at::kInt) || starts->numel() != batch + 1) return std::nullopt;
        most_q = max_q && *max_q < rows ? *max_q : rows;
    } else {
        if (rows % batch != 0) return std::nullopt;
        most_q = rows / batch;
        if (max_q && *max_q != most_q) return std::nullopt;
    }
    int64_t keys = table.size(1) * c.c.page_size;
    if (max_keys && *max_keys < keys) keys = *max_keys;
    if (most_q <= 0 || keys < 0) return std::nullopt;
    at::NoGradGuard no_grad;
    Tensor out = at::empty(q.sizes(), q.options().memory_format(at::MemoryFormat::Contiguous));
    const size_t need = mxq_kv_attention_workspace_bytes(&c.c, batch, rows, (int32_t)most_q, (int32_t)heads, keys);
    Tensor ws;
    if (need) ws = scratch((int64_t)need, q);
    if (mxq_kv_attention(c.raw(), q.const_data_ptr(), rows, rows > 1 ? q.stride(0) : 0, heads > 1 ? q.stride(1) : 0, (int32_t)heads, batch,
                         starts ? starts->const_data_ptr<int32_t>() : nullptr, (int32_t)most_q, lens.const_data_ptr<int32_t>(), keys,
                         table.const_data_ptr<int32_t>(), table.size(1),
                         scale ? (float)*scale : 1.0f / std::sqrt((float)c.c.head_dim), (int32_t)window, 1, out.mutable_data_ptr(), nullptr,
                         need ? ws.mutable_data_ptr() : nullptr, need, stream_of(q)) != MXQ_OK)
        return std::nullopt;
    return out;
}

}  // namespace

PYBIND11_MODULE(_ops, m) {
    m.doc() = "The plain cases of the operators in ops.py; None (or False) for any other case.";
    py::class_<Cache>(m, "Cache");
    m.def("linear", &linear);
    m.def("linear_ste", &linear_ste);
    m.def("swiglu", &swiglu);
    m.def("cache", &cache);
    m.def("kv_append", &kv_append);
    m.def("kv_read", &kv_read);
    m.def("kv_attention", &kv_attention);
}
