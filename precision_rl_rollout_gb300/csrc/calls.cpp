// calls.cpp -- the rollout step's calls (rotary positions, the append, paged
// attention, verification) and the trainer's losses (log-probabilities from hidden
// states, distillation) from torch tensors to the C ABI, as a Python module.
// A decode step makes these calls with a few microseconds of GPU work behind each;
// checked and marshalled in Python they took 11 to 23 us of host time, here 4 to
// 11 (Grace; the launches themselves are 3 to 6 of it).  Everything they refuse is
// refused with ValueError before any CUDA call; a status of the C ABI becomes the
// binding's Fp8rlError.  The module links to no part of the library: bind() is given
// the addresses of its functions.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
#include <sstream>
#include <stdexcept>
#include <string>

#include "fp8rl.h"

namespace {

using at::Tensor;

struct Functions {
    decltype(&fp8rl_rope) rope;
    decltype(&fp8rl_rope_append_paged) rope_append_paged;
    decltype(&fp8rl_attn_paged) attn_paged;
    decltype(&fp8rl_attn_paged_workspace_bytes) attn_workspace;
    decltype(&fp8rl_spec_verify) spec_verify;
    decltype(&fp8rl_linear_logp) linear_logp;
    decltype(&fp8rl_linear_logp_workspace_bytes) linear_logp_workspace;
    decltype(&fp8rl_linear_logp_backward) linear_logp_backward;
    decltype(&fp8rl_linear_logp_backward_workspace_bytes) linear_logp_backward_workspace;
    decltype(&fp8rl_distill_topk) distill_topk;
    decltype(&fp8rl_distill_topk_backward) distill_topk_backward;
} fn = {};
PyObject* status_error = nullptr;                 // binding.Fp8rlError

struct Status {                                   // a status other than FP8RL_OK
    int rc;
    const char* where;
};

[[noreturn]] void refuse(const char* name, const Tensor& t, const std::string& want) {
    std::ostringstream s;
    s << name << ": expected " << want << ", got " << t.dtype() << ' ' << t.sizes() << " strides " << t.strides()
      << " on " << t.device();
    throw std::invalid_argument(s.str());
}

const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw std::invalid_argument(std::string(name) + ": expected a tensor");
    return THPVariable_Unpack(o);
}
int64_t integer(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw std::invalid_argument(std::string(name) + ": expected an integer");
    }
    return v;
}
bool truth(PyObject* o) { return PyObject_IsTrue(o) == 1; }

// The device of a call: its first tensor's.
c10::Device cuda_device(const Tensor& t, const char* name) {
    if (!t.is_cuda()) refuse(name, t, "a CUDA tensor");
    return t.device();
}
void dense(const Tensor& t, at::ScalarType type, at::IntArrayRef shape, c10::Device dev, const char* name) {
    if (t.scalar_type() != type || t.sizes() != shape || t.device() != dev || !t.is_contiguous()) {
        std::ostringstream s;
        s << "contiguous " << type << ' ' << shape << " on " << dev;
        refuse(name, t, s.str());
    }
}
// bf16 heads of contiguous values.
void heads(const Tensor& t, int64_t dim, c10::Device dev, const char* name) {
    if (t.scalar_type() != at::kBFloat16 || t.dim() != dim || t.device() != dev ||
        (t.stride(dim - 1) != 1 && t.size(dim - 1) > 1))
        refuse(name, t, "bfloat16 on the call's device, " + std::to_string(dim) + "-D with contiguous head values");
}
template <typename T>
T* ptr(const Tensor& t) {
    return static_cast<T*>(t.data_ptr());
}

// Pools [pages, page_size, kv_heads, head_dim].
fp8rl_paged_kv paged_kv(PyObject* ko, PyObject* vo, PyObject* kso, PyObject* vso, c10::Device dev) {
    const Tensor &K = tensor(ko, "K"), &V = tensor(vo, "V");
    if (K.dim() != 4 || K.device() != dev || K.stride(3) != 1 ||
        (K.scalar_type() != at::kBFloat16 && K.scalar_type() != at::kByte))
        refuse("K", K, "[pages, page_size, kv_heads, head_dim] on the call's device, bfloat16 values or uint8 E4M3 "
                       "codes, with contiguous head values");
    if (V.scalar_type() != K.scalar_type() || V.sizes() != K.sizes() || V.strides() != K.strides() || V.device() != dev)
        refuse("V", V, "K's type, shape, strides and device");
    fp8rl_paged_kv kv = {};
    kv.K = K.data_ptr(), kv.V = V.data_ptr();
    kv.dtype = FP8RL_KV_BF16;
    if (K.scalar_type() == at::kByte) {
        kv.dtype = FP8RL_KV_E4M3;
        if (kso == Py_None || vso == Py_None)
            throw std::invalid_argument("k_scale, v_scale: an E4M3 cache needs its scales, float32 [1]");
        const Tensor &ks = tensor(kso, "k_scale"), &vs = tensor(vso, "v_scale");
        dense(ks, at::kFloat, {1}, dev, "k_scale");
        dense(vs, at::kFloat, {1}, dev, "v_scale");
        kv.k_scale = ptr<float>(ks), kv.v_scale = ptr<float>(vs);
    }
    kv.num_pages = K.size(0), kv.page_size = K.size(1), kv.kv_heads = K.size(2), kv.head_dim = K.size(3);
    kv.page_stride = K.stride(0), kv.token_stride = K.stride(1), kv.head_stride = K.stride(2);
    return kv;
}

// The call's device and stream (None: torch's current one there; else the raw stream),
// made current while it lasts, so that what the call allocates is of its own stream's
// memory: a block of another stream's can have work of that stream still queued on it.
// Outputs on a given stream are recorded on the caller's, which will read them.
class Launch {
public:
    Launch(PyObject* o, c10::Device dev)
        : caller_(c10::cuda::getCurrentCUDAStream(dev.index())), stream_(pick(o, dev, caller_)), guard_(stream_) {}
    void* stream() const { return stream_.stream(); }
    Tensor empty(at::IntArrayRef shape, const at::TensorOptions& options) const {
        Tensor t = at::empty(shape, options);
        if (stream_.stream() != caller_.stream()) t.record_stream(caller_.unwrap());
        return t;
    }

private:
    static c10::cuda::CUDAStream pick(PyObject* o, c10::Device dev, c10::cuda::CUDAStream caller) {
        if (o == Py_None) return caller;
        void* const raw = PyLong_AsVoidPtr(o);
        if (!raw && PyErr_Occurred()) {
            PyErr_Clear();
            throw std::invalid_argument("stream: expected a raw stream");
        }
        return c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(raw), dev.index());
    }
    c10::cuda::CUDAStream caller_, stream_;
    c10::cuda::CUDAStreamGuard guard_;
};

// While it lasts other Python threads run: a launch waits where the driver's queue is
// full or a kernel is loaded for its first call.  The caller holds the tensors.
class Released {
public:
    Released() : state_(PyEval_SaveThread()) {}
    ~Released() { PyEval_RestoreThread(state_); }
    Released(const Released&) = delete;
    Released& operator=(const Released&) = delete;

private:
    PyThreadState* state_;
};
template <typename F, typename... Args>
int unlocked(F f, Args... args) {
    const Released released;
    return f(args...);
}

// Table [max_pos, R] and positions [T].
void check_table(const Tensor& positions, const Tensor& table, int64_t T, c10::Device dev) {
    dense(positions, at::kInt, {T}, dev, "positions");
    if (table.scalar_type() != at::kFloat || table.dim() != 2 || table.device() != dev || !table.is_contiguous())
        refuse("table", table, "contiguous float32 [max_pos, R] on the call's device");
}

// Y given, or new: [like X].
Tensor output_like(const Launch& launch, PyObject* o, const Tensor& X, const char* name) {
    if (o == Py_None) return launch.empty(X.sizes(), X.options());
    const Tensor& Y = tensor(o, name);
    heads(Y, X.dim(), X.device(), name);
    if (Y.sizes() != X.sizes()) refuse(name, Y, "the input's shape");
    return Y;
}
Tensor output(const Launch& launch, PyObject* o, at::IntArrayRef shape, at::ScalarType type, const Tensor& like,
              const char* name) {
    if (o == Py_None) return launch.empty(shape, like.options().dtype(type));
    const Tensor& t = tensor(o, name);
    dense(t, type, shape, like.device(), name);
    return t;
}

// ------------------------------------------------------------------ the calls

// X, positions, table, interleaved, inverse, Y, stream
PyObject* rope(PyObject* const* a) {
    const Tensor& X = tensor(a[0], "X");
    const c10::Device dev = cuda_device(X, "X");
    heads(X, 3, dev, "X");
    const Tensor &positions = tensor(a[1], "positions"), &table = tensor(a[2], "table");
    const int64_t T = X.size(0), H = X.size(1), D = X.size(2);
    check_table(positions, table, T, dev);
    const Launch launch(a[6], dev);
    const Tensor Y = output_like(launch, a[5], X, "Y");
    const unsigned flags = (truth(a[3]) ? FP8RL_ROPE_INTERLEAVED : 0) | (truth(a[4]) ? FP8RL_ROPE_INVERSE : 0);
    const int rc = unlocked(fn.rope, ptr<uint16_t>(X), T, H, D, X.stride(0), X.stride(1), ptr<int32_t>(positions),
                            ptr<float>(table), table.size(0), table.size(1), flags, ptr<uint16_t>(Y), Y.stride(0),
                            Y.stride(1), launch.stream());
    if (rc) throw Status{rc, "fp8rl_rope"};
    return THPVariable_Wrap(Y);
}

// q, k, v, positions, table, K, V, slots, k_scale, v_scale, interleaved, q_out, stream
PyObject* rope_append_paged(PyObject* const* a) {
    const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const c10::Device dev = cuda_device(q, "q");
    heads(q, 3, dev, "q");
    heads(k, 3, dev, "k");
    heads(v, 3, dev, "v");
    const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2);
    const fp8rl_paged_kv kv = paged_kv(a[5], a[6], a[8], a[9], dev);
    const int64_t shape[3] = {T, kv.kv_heads, D};
    if (kv.head_dim != D || k.sizes() != at::IntArrayRef(shape, 3) || v.sizes() != k.sizes())
        throw std::invalid_argument("k and v must be [T, kv_heads, D] with the cache's heads and q's T and D");
    const Tensor& slots = tensor(a[7], "slots");
    dense(slots, at::kLong, {T}, dev, "slots");
    const int32_t* positions = nullptr;
    const float* rows = nullptr;
    int64_t max_pos = 0, R = 0;
    if (a[4] != Py_None) {
        const Tensor &p = tensor(a[3], "positions"), &table = tensor(a[4], "table");
        check_table(p, table, T, dev);
        positions = ptr<int32_t>(p), rows = ptr<float>(table), max_pos = table.size(0), R = table.size(1);
    }
    const Launch launch(a[12], dev);
    const Tensor out = output_like(launch, a[11], q, "q_out");
    const int rc = unlocked(fn.rope_append_paged, ptr<uint16_t>(q), Hq, q.stride(0), q.stride(1), ptr<uint16_t>(k),
                            k.stride(0), k.stride(1), ptr<uint16_t>(v), v.stride(0), v.stride(1), T, positions, rows,
                            max_pos, R, truth(a[10]) ? FP8RL_ROPE_INTERLEAVED : 0, ptr<uint16_t>(out), out.stride(0),
                            out.stride(1), &kv, ptr<int64_t>(slots), launch.stream());
    if (rc) throw Status{rc, "fp8rl_rope_append_paged"};
    return THPVariable_Wrap(out);
}

// q, K, V, block_table, seq_lens, max_len, scale, window, k_scale, v_scale, o, lse, want_lse, workspace, stream
PyObject* attn_paged(PyObject* const* a) {
    const Tensor& q = tensor(a[0], "q");
    const c10::Device dev = cuda_device(q, "q");
    heads(q, 4, dev, "q");
    const int64_t B = q.size(0), Lq = q.size(1), Hq = q.size(2), D = q.size(3);
    const fp8rl_paged_kv kv = paged_kv(a[1], a[2], a[8], a[9], dev);
    if (kv.head_dim != D) throw std::invalid_argument("q and the cache must have the same head width");
    const int64_t max_len = integer(a[5], "max_len"), window = integer(a[7], "window");
    const Tensor &table = tensor(a[3], "block_table"), &lens = tensor(a[4], "seq_lens");
    if (table.scalar_type() != at::kInt || table.dim() != 2 || table.device() != dev || table.size(0) != B ||
        (table.stride(1) != 1 && table.size(1) > 1) || table.size(1) * kv.page_size < max_len)
        refuse("block_table", table, "int32 [B, columns] on the call's device, with contiguous rows that cover max_len tokens");
    dense(lens, at::kInt, {B}, dev, "seq_lens");
    double scale = 0.0;
    if (a[6] == Py_None) {
        scale = 1.0 / std::sqrt((double)D);
    } else {
        scale = PyFloat_AsDouble(a[6]);
        if (scale == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            throw std::invalid_argument("scale: expected a number");
        }
    }
    const Launch launch(a[14], dev);
    const Tensor o = output(launch, a[10], q.sizes(), at::kBFloat16, q, "o");
    Tensor lse, workspace;
    if (a[11] != Py_None || truth(a[12])) lse = output(launch, a[11], q.sizes().slice(0, 3), at::kFloat, q, "lse");
    if (a[13] != Py_None) {
        workspace = tensor(a[13], "workspace");
        if (workspace.device() != dev || !workspace.is_contiguous())
            refuse("workspace", workspace, "a contiguous tensor on the call's device");
    } else if (const size_t need = fn.attn_workspace(B, Lq, Hq, kv.kv_heads, D, max_len)) {
        workspace = at::empty({(int64_t)need}, q.options().dtype(at::kByte));
    }
    const int rc = unlocked(fn.attn_paged, ptr<uint16_t>(q), B, Lq, Hq, q.stride(0), q.stride(1), q.stride(2), &kv,
                            ptr<int32_t>(table), B == 1 ? table.size(1) : table.stride(0), ptr<int32_t>(lens), max_len,
                            window, (float)scale, ptr<uint16_t>(o), lse.defined() ? ptr<float>(lse) : nullptr,
                            workspace.defined() ? workspace.data_ptr() : nullptr,
                            workspace.defined() ? workspace.nbytes() : 0, launch.stream());
    if (rc) throw Status{rc, "fp8rl_attn_paged"};
    if (!lse.defined()) return THPVariable_Wrap(o);
    return Py_BuildValue("(NN)", THPVariable_Wrap(o), THPVariable_Wrap(lse));
}

// P, drafts, u, noise, Q, draft_lens, tokens, accepted, stream
PyObject* spec_verify(PyObject* const* a) {
    const Tensor& P = tensor(a[0], "P");
    const c10::Device dev = cuda_device(P, "P");
    const at::ScalarType type = P.scalar_type();
    if ((type != at::kFloat && type != at::kBFloat16) || P.dim() != 3 || (P.stride(2) != 1 && P.size(2) > 1))
        refuse("P", P, "[B, K + 1, V] float32 or bfloat16 with contiguous rows");
    const int64_t B = P.size(0), K = P.size(1) - 1, V = P.size(2);
    const void* qp = nullptr;
    int64_t q_seq = 0, q_step = 0;
    if (a[4] != Py_None) {
        const Tensor& Q = tensor(a[4], "Q");
        const int64_t shape[3] = {B, K, V};
        if (Q.scalar_type() != type || Q.sizes() != at::IntArrayRef(shape, 3) || Q.device() != dev ||
            (Q.stride(2) != 1 && V > 1))
            refuse("Q", Q, "[B, K, V] of P's type and device with contiguous rows");
        qp = Q.data_ptr(), q_seq = Q.stride(0), q_step = Q.stride(1);
    }
    const Tensor &drafts = tensor(a[1], "drafts"), &u = tensor(a[2], "u"), &noise = tensor(a[3], "noise");
    dense(drafts, at::kInt, {B, K}, dev, "drafts");
    dense(u, at::kFloat, {B, K}, dev, "u");
    if (noise.scalar_type() != at::kFloat || noise.dim() != 2 || noise.size(0) != B || noise.size(1) != V ||
        noise.device() != dev || (noise.stride(1) != 1 && V > 1))
        refuse("noise", noise, "float32 [B, V] with contiguous rows on P's device");
    const int32_t* lens = nullptr;
    if (a[5] != Py_None) {
        const Tensor& t = tensor(a[5], "draft_lens");
        dense(t, at::kInt, {B}, dev, "draft_lens");
        lens = ptr<int32_t>(t);
    }
    const Launch launch(a[8], dev);
    const Tensor tokens = output(launch, a[6], {B, K + 1}, at::kInt, P, "tokens");
    const Tensor accepted = output(launch, a[7], {B}, at::kInt, P, "accepted");
    const int rc = unlocked(fn.spec_verify, P.data_ptr(), P.stride(0), P.stride(1), qp, q_seq, q_step,
                            type == at::kFloat ? FP8RL_PROB_F32 : FP8RL_PROB_BF16, ptr<int32_t>(drafts), lens,
                            ptr<float>(u), ptr<float>(noise), noise.stride(0), B, K, V, ptr<int32_t>(tokens),
                            ptr<int32_t>(accepted), launch.stream());
    if (rc) throw Status{rc, "fp8rl_spec_verify"};
    return Py_BuildValue("(NN)", THPVariable_Wrap(tokens), THPVariable_Wrap(accepted));
}

// ------------------------------------------------------------------ the trainer's losses

double number(PyObject* o, const char* name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw std::invalid_argument(std::string(name) + ": expected a number");
    }
    return v;
}
// A matrix with contiguous rows.
void matrix(const Tensor& t, at::ScalarType type, int64_t cols, c10::Device dev, const char* name) {
    if (t.scalar_type() != type || t.dim() != 2 || t.device() != dev || (cols >= 0 && t.size(1) != cols) ||
        (t.stride(1) != 1 && t.size(1) > 1)) {
        std::ostringstream s;
        s << type << " [rows, " << (cols >= 0 ? std::to_string(cols) : std::string("columns"))
          << "] with contiguous rows on " << dev;
        refuse(name, t, s.str());
    }
}
// Its row pitch; a single row's stride says nothing.
int64_t pitch(const Tensor& t, int64_t multiple) {
    return t.size(0) > 1 ? t.stride(0) : (t.size(1) + multiple - 1) / multiple * multiple;
}
const float* vector_or_null(PyObject* o, int64_t n, c10::Device dev, const char* name) {
    if (o == Py_None) return nullptr;
    const Tensor& t = tensor(o, name);
    dense(t, at::kFloat, {n}, dev, name);
    return ptr<float>(t);
}
Tensor scratch(PyObject* o, size_t need, const Tensor& like) {
    if (o != Py_None) {
        const Tensor& t = tensor(o, "workspace");
        if (t.device() != like.device() || !t.is_contiguous())
            refuse("workspace", t, "a contiguous tensor on the call's device");
        return t;
    }
    return at::empty({(int64_t)need}, like.options().dtype(at::kByte));
}

struct Head {                                     // hidden states, output matrix, targets
    const Tensor &H, &W, &targets;
    int64_t M, V, K;
    c10::Device dev;
    explicit Head(PyObject* const* a)
        : H(tensor(a[0], "H")), W(tensor(a[1], "W")), targets(tensor(a[2], "targets")), dev(cuda_device(H, "H")) {
        matrix(H, at::kBFloat16, -1, dev, "H");
        matrix(W, at::kBFloat16, H.size(1), dev, "W");
        M = H.size(0), K = H.size(1), V = W.size(0);
        dense(targets, at::kInt, {M}, dev, "targets");
    }
};

// H, W, targets, scale, logp, lse, entropy, want_entropy, workspace, stream
PyObject* linear_logp(PyObject* const* a) {
    const Head h(a);
    const float scale = (float)number(a[3], "scale");
    const Launch launch(a[9], h.dev);
    const Tensor logp = output(launch, a[4], {h.M}, at::kFloat, h.H, "logp");
    const Tensor lse = output(launch, a[5], {h.M}, at::kFloat, h.H, "lse");
    Tensor entropy;
    if (a[6] != Py_None || truth(a[7])) entropy = output(launch, a[6], {h.M}, at::kFloat, h.H, "entropy");
    const Tensor ws = scratch(a[8], fn.linear_logp_workspace(h.M, h.V, h.K), h.H);
    const int rc = unlocked(fn.linear_logp, ptr<uint16_t>(h.H), pitch(h.H, 8), ptr<uint16_t>(h.W), pitch(h.W, 8),
                            ptr<int32_t>(h.targets), h.M, h.V, h.K, scale, ptr<float>(logp), ptr<float>(lse),
                            entropy.defined() ? ptr<float>(entropy) : nullptr, ws.data_ptr(), ws.nbytes(),
                            launch.stream());
    if (rc) throw Status{rc, "fp8rl_linear_logp"};
    if (!entropy.defined()) return Py_BuildValue("(NN)", THPVariable_Wrap(logp), THPVariable_Wrap(lse));
    return Py_BuildValue("(NNN)", THPVariable_Wrap(logp), THPVariable_Wrap(lse), THPVariable_Wrap(entropy));
}

// H, W, targets, lse, g_logp, entropy, g_entropy, scale, dH, dW, want_dH, want_dW, workspace, stream
PyObject* linear_logp_backward(PyObject* const* a) {
    const Head h(a);
    const Tensor &lse = tensor(a[3], "lse"), &g = tensor(a[4], "g_logp");
    dense(lse, at::kFloat, {h.M}, h.dev, "lse");
    dense(g, at::kFloat, {h.M}, h.dev, "g_logp");
    const float* entropy = vector_or_null(a[5], h.M, h.dev, "entropy");
    const float* ge = vector_or_null(a[6], h.M, h.dev, "g_entropy");
    if (a[6] != Py_None && a[5] == Py_None)
        throw std::invalid_argument("g_entropy: the gradient of the entropy needs the forward's entropy");
    const float scale = (float)number(a[7], "scale");
    const Launch launch(a[13], h.dev);
    Tensor dH, dW;
    if (a[8] != Py_None || truth(a[10])) dH = output(launch, a[8], {h.M, h.K}, at::kBFloat16, h.H, "dH");
    if (a[9] != Py_None || truth(a[11])) dW = output(launch, a[9], {h.V, h.K}, at::kBFloat16, h.H, "dW");
    if (!dH.defined() && !dW.defined()) throw std::invalid_argument("neither dH nor dW is wanted");
    const Tensor ws = scratch(a[12], fn.linear_logp_backward_workspace(h.M, h.V, h.K), h.H);
    const int rc = unlocked(fn.linear_logp_backward, ptr<uint16_t>(h.H), pitch(h.H, 8), ptr<uint16_t>(h.W),
                            pitch(h.W, 8), ptr<int32_t>(h.targets), ptr<float>(lse), entropy, ptr<float>(g), ge, h.M,
                            h.V, h.K, scale, dH.defined() ? ptr<uint16_t>(dH) : nullptr,
                            dW.defined() ? ptr<uint16_t>(dW) : nullptr, ws.data_ptr(), ws.nbytes(), launch.stream());
    if (rc) throw Status{rc, "fp8rl_linear_logp_backward"};
    auto wrap = [](const Tensor& t) {
        if (t.defined()) return THPVariable_Wrap(t);
        Py_INCREF(Py_None);
        return Py_None;
    };
    return Py_BuildValue("(NN)", wrap(dH), wrap(dW));
}

struct Logits {                                   // a student's logits and a teacher's entries
    const Tensor &X, &indices, &T;
    int64_t M, V, k, multiple;
    int dtype;
    c10::Device dev;
    explicit Logits(PyObject* const* a)
        : X(tensor(a[0], "X")), indices(tensor(a[1], "indices")), T(tensor(a[2], "T")), dev(cuda_device(X, "X")) {
        if (X.scalar_type() != at::kFloat && X.scalar_type() != at::kBFloat16)
            refuse("X", X, "float32 or bfloat16 logits");
        matrix(X, X.scalar_type(), -1, dev, "X");
        M = X.size(0), V = X.size(1);
        if (indices.dim() != 2) refuse("indices", indices, "int32 [M, k]");
        k = indices.size(1);
        dense(indices, at::kInt, {M, k}, dev, "indices");
        dense(T, at::kFloat, {M, k}, dev, "T");
        dtype = X.scalar_type() == at::kFloat ? FP8RL_LOGITS_F32 : FP8RL_LOGITS_BF16;
        multiple = X.scalar_type() == at::kFloat ? 4 : 8;
    }
};

// X, indices, T, teacher_lse, rest, scale, loss, lse, rest_lse, stream
PyObject* distill_topk(PyObject* const* a) {
    const Logits x(a);
    const float* teacher = vector_or_null(a[3], x.M, x.dev, "teacher_lse");
    const bool rest = a[8] != Py_None || truth(a[4]);
    if (rest && a[3] == Py_None) throw std::invalid_argument("rest: what the entries leave needs teacher_lse");
    const float scale = (float)number(a[5], "scale");
    const Launch launch(a[9], x.dev);
    const Tensor loss = output(launch, a[6], {x.M}, at::kFloat, x.X, "loss");
    const Tensor lse = output(launch, a[7], {x.M}, at::kFloat, x.X, "lse");
    Tensor rest_lse;
    if (rest) rest_lse = output(launch, a[8], {x.M}, at::kFloat, x.X, "rest_lse");
    const int rc = unlocked(fn.distill_topk, x.X.data_ptr(), pitch(x.X, x.multiple), x.dtype, ptr<int32_t>(x.indices),
                            ptr<float>(x.T), teacher, x.M, x.V, x.k, scale, ptr<float>(loss), ptr<float>(lse),
                            rest ? ptr<float>(rest_lse) : nullptr, launch.stream());
    if (rc) throw Status{rc, "fp8rl_distill_topk"};
    if (!rest) return Py_BuildValue("(NN)", THPVariable_Wrap(loss), THPVariable_Wrap(lse));
    return Py_BuildValue("(NNN)", THPVariable_Wrap(loss), THPVariable_Wrap(lse), THPVariable_Wrap(rest_lse));
}

// X, indices, T, lse, g_loss, teacher_lse, rest_lse, scale, dX, stream
PyObject* distill_topk_backward(PyObject* const* a) {
    const Logits x(a);
    const Tensor &lse = tensor(a[3], "lse"), &g = tensor(a[4], "g_loss");
    dense(lse, at::kFloat, {x.M}, x.dev, "lse");
    dense(g, at::kFloat, {x.M}, x.dev, "g_loss");
    const float* teacher = vector_or_null(a[5], x.M, x.dev, "teacher_lse");
    const float* rest = vector_or_null(a[6], x.M, x.dev, "rest_lse");
    if (a[6] != Py_None && a[5] == Py_None) throw std::invalid_argument("rest_lse: what the entries leave needs teacher_lse");
    const float scale = (float)number(a[7], "scale");
    const Launch launch(a[9], x.dev);
    Tensor dX;
    if (a[8] == Py_None) {                        // rows padded to whole 16 bytes
        const int64_t cols = (x.V + x.multiple - 1) / x.multiple * x.multiple;
        dX = launch.empty({x.M, cols}, x.X.options());
        if (cols != x.V) dX = dX.narrow(1, 0, x.V);
    } else {
        dX = tensor(a[8], "dX");
        matrix(dX, x.X.scalar_type(), x.V, x.dev, "dX");
        if (dX.size(0) != x.M) refuse("dX", dX, "X's shape");
    }
    const int rc = unlocked(fn.distill_topk_backward, x.X.data_ptr(), pitch(x.X, x.multiple), x.dtype,
                            ptr<int32_t>(x.indices), ptr<float>(x.T), teacher, ptr<float>(lse), rest, ptr<float>(g),
                            x.M, x.V, x.k, scale, dX.data_ptr(), pitch(dX, x.multiple), launch.stream());
    if (rc) throw Status{rc, "fp8rl_distill_topk_backward"};
    return THPVariable_Wrap(dX);
}

// No C++ exception passes into Python.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    try {
        if (n != N) throw std::invalid_argument("expected " + std::to_string(N) + " arguments");
        if (!status_error || !fn.distill_topk_backward && (F == linear_logp || F == linear_logp_backward ||
                                                           F == distill_topk || F == distill_topk_backward))
            throw std::runtime_error("bind() has not been called");
        return F(args);
    } catch (const Status& s) {
        if (PyObject* e = PyObject_CallFunction(status_error, "is", s.rc, s.where)) {
            PyErr_SetObject(status_error, e);
            Py_DECREF(e);
        }
    } catch (const std::invalid_argument& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// Addresses of fp8rl_rope, _rope_append_paged, _attn_paged, _attn_paged_workspace_bytes, _spec_verify; Fp8rlError
PyObject* bind(PyObject*, PyObject* args) {
    unsigned long long f[5];
    PyObject* error = nullptr;
    if (!PyArg_ParseTuple(args, "KKKKKO", &f[0], &f[1], &f[2], &f[3], &f[4], &error)) return nullptr;
    fn.rope = reinterpret_cast<decltype(fn.rope)>(f[0]);
    fn.rope_append_paged = reinterpret_cast<decltype(fn.rope_append_paged)>(f[1]);
    fn.attn_paged = reinterpret_cast<decltype(fn.attn_paged)>(f[2]);
    fn.attn_workspace = reinterpret_cast<decltype(fn.attn_workspace)>(f[3]);
    fn.spec_verify = reinterpret_cast<decltype(fn.spec_verify)>(f[4]);
    Py_INCREF(error);
    Py_XSETREF(status_error, error);
    Py_RETURN_NONE;
}

// Addresses of fp8rl_linear_logp, its workspace query, _backward, its query, fp8rl_distill_topk, _backward
PyObject* bind_losses(PyObject*, PyObject* args) {
    unsigned long long f[6];
    if (!PyArg_ParseTuple(args, "KKKKKK", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5])) return nullptr;
    fn.linear_logp = reinterpret_cast<decltype(fn.linear_logp)>(f[0]);
    fn.linear_logp_workspace = reinterpret_cast<decltype(fn.linear_logp_workspace)>(f[1]);
    fn.linear_logp_backward = reinterpret_cast<decltype(fn.linear_logp_backward)>(f[2]);
    fn.linear_logp_backward_workspace = reinterpret_cast<decltype(fn.linear_logp_backward_workspace)>(f[3]);
    fn.distill_topk = reinterpret_cast<decltype(fn.distill_topk)>(f[4]);
    fn.distill_topk_backward = reinterpret_cast<decltype(fn.distill_topk_backward)>(f[5]);
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef fast(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {fast<rope, 7>("rope"), fast<rope_append_paged, 13>("rope_append_paged"),
                         fast<attn_paged, 15>("attn_paged"), fast<spec_verify, 9>("spec_verify"),
                         fast<linear_logp, 10>("linear_logp"),
                         fast<linear_logp_backward, 14>("linear_logp_backward"),
                         fast<distill_topk, 10>("distill_topk"),
                         fast<distill_topk_backward, 10>("distill_topk_backward"),
                         {"bind", bind, METH_VARARGS, nullptr}, {"bind_losses", bind_losses, METH_VARARGS, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
