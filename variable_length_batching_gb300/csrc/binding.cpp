// Compiled argument marshalling of the attention path's calls (nt.py's
// functions of the same names): tensors in, C-ABI calls out.  A decoding step
// makes these calls for microseconds of device work each; checking and
// passing their arguments from Python took several times as long as the
// kernels (19 us for a 3 us norm and rotation).  It computes nothing and
// links no CUDA code: the C functions' addresses come from the loaded libnt.
//
// Every function takes its arguments by position (None for an absent tensor)
// and returns (status, outputs...).  Mismatched tensors raise ValueError here;
// what the C call refuses comes back as its status.  Outputs and workspaces
// that the caller does not give are allocated on the call's stream.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <optional>
#include <string>

#include "../../include/nt.h"

namespace {

decltype(&nt_qk_norm_rope) f_rope;
decltype(&nt_qk_norm_rope_bwd) f_rope_bwd;
decltype(&nt_qk_norm_rope_bwd_workspace_bytes) f_rope_bwd_ws;
decltype(&nt_paged_write) f_write;
decltype(&nt_paged_copy) f_copy;
decltype(&nt_paged_attn) f_attn;
decltype(&nt_paged_attn_workspace_bytes) f_attn_ws;
decltype(&nt_paged_write_slots) f_write_slots;
decltype(&nt_paged_resize) f_resize;
decltype(&nt_draft_tree) f_tree;
decltype(&nt_paged_keep) f_keep;
decltype(&nt_paged_tree_attn) f_tree_attn;
decltype(&nt_paged_tree_attn_workspace_bytes) f_tree_attn_ws;

// A mismatch: ValueError with this text.
struct Mismatch {
  std::string text;
};
[[noreturn]] void refuse(std::string text) { throw Mismatch{std::move(text)}; }

using T = at::Tensor;

const T& none() {
  static const T t;
  return t;
}
// An argument that is a tensor or None.
const T& tensor(PyObject* o, const char* name) {
  if (o == Py_None) return none();
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
const T& need(PyObject* o, const char* name) {
  const T& t = tensor(o, name);
  if (!t.defined()) refuse(std::string(name) + " is needed");
  return t;
}
const char* type_name(at::ScalarType t) { return c10::toString(t); }

void on_device(const T& t, int index, const char* name) {
  if (!t.is_cuda() || t.get_device() != index)
    refuse(std::string(name) + " is on " + t.device().str() + ", expected cuda:" + std::to_string(index));
}
// Address of a contiguous tensor on the device (NULL for none).
void* flat(const T& t, int index, at::ScalarType type, const char* name) {
  if (!t.defined()) return nullptr;
  on_device(t, index, name);
  if (t.scalar_type() != type) refuse(std::string(name) + " must be " + type_name(type));
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  return t.data_ptr();
}

// Packed tokens (T, H, d) whose heads are contiguous within a token; tokens
// may be any stride apart.
struct Tokens {
  void* p = nullptr;
  int64_t stride = 0;
};
Tokens tokens(const T& t, int index, at::ScalarType type, const char* name) {
  if (!t.defined()) return {};
  on_device(t, index, name);
  if (t.scalar_type() != type) refuse(std::string(name) + " must be " + type_name(type));
  if (t.dim() != 3) refuse(std::string(name) + " must be (tokens, heads, d)");
  const int64_t n = t.size(0), H = t.size(1), d = t.size(2);
  if (n * H * d > 0 && ((d > 1 && t.stride(2) != 1) || (H > 1 && t.stride(1) != d)))
    refuse(std::string(name) + ": the heads of a token must be contiguous");
  return {t.data_ptr(), n > 1 ? t.stride(0) : H * d};
}

int32_t dtype_of(at::ScalarType t) {
  if (t == at::kBFloat16) return NT_BF16;
  if (t == at::kFloat) return NT_F32;
  refuse(std::string("unsupported dtype ") + type_name(t));
}

int32_t flag(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

// The call's device and stream, current while it lasts: the device's current
// stream, or the handle given.
struct Call {
  c10::cuda::CUDAGuard device;
  std::optional<c10::cuda::CUDAStreamGuard> on;
  cudaStream_t stream;
  Call(int index, PyObject* handle) : device(static_cast<c10::DeviceIndex>(index)) {
    if (handle == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(index).stream();
    } else {
      void* h = PyLong_AsVoidPtr(handle);
      if (!h && PyErr_Occurred()) throw python_error();
      stream = static_cast<cudaStream_t>(h);
      on.emplace(h ? c10::cuda::getStreamFromExternal(stream, index) : c10::cuda::getDefaultCUDAStream(index));
    }
  }
};

// A new contiguous tensor, without the dispatcher's way to the allocator.
T fresh(at::IntArrayRef sizes, at::ScalarType type, int index) {
  return T(at::detail::empty_cuda(sizes, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(index)),
                                  std::nullopt));
}
// n elements of another type over a part of a tensor's memory.
T part(const T& all, int64_t at, at::IntArrayRef sizes, at::ScalarType type) {
  T t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(),
                                                 c10::scalarTypeToTypeMeta(type));
  c10::TensorImpl* impl = t.unsafeGetTensorImpl();
  impl->set_storage_offset(at / (int64_t)c10::elementSize(type));
  impl->set_sizes_contiguous(sizes);
  return t;
}
T like(const T& t) { return fresh(t.sizes(), t.scalar_type(), t.get_device()); }
T bytes(size_t n, const T& t) { return fresh({(int64_t)n}, at::kByte, t.get_device()); }
void* data(const T& t) { return t.defined() ? t.data_ptr() : nullptr; }
bool same_shape(const T& a, const T& b) { return a.defined() == b.defined() && (!a.defined() || a.sizes() == b.sizes()); }

// The interpreter's lock is not held across a C call: a launch waits where the
// device's queue is full, possibly for work that needs the lock.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename F, typename... A>
int unlocked(F f, A... args) {
  const Unlocked u;
  return f(args...);
}

PyObject* result(int status, std::initializer_list<const T*> outs) {
  PyObject* r = PyTuple_New(1 + outs.size());
  if (!r) throw python_error();
  PyTuple_SET_ITEM(r, 0, PyLong_FromLong(status));
  Py_ssize_t i = 1;
  for (const T* t : outs) {
    PyObject* o;
    if (t->defined()) {
      o = THPVariable_Wrap(*t);
    } else {
      Py_INCREF(Py_None);
      o = Py_None;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

void arity(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) refuse("expected " + std::to_string(want) + " arguments, got " + std::to_string(got));
}

// What the rope calls share: sizes, positions, gammas.
struct Rope {
  int index;
  at::ScalarType type;
  int64_t n, H_q, H_k, d;
  const int32_t *cu, *pos0, *positions;
  int32_t B;
  const uint64_t* turns;
  int32_t rot;
  const float *qg, *kg;
  Rope(const T& q, const T& k, const T& turns_, const T& cu_, const T& positions_, const T& pos0_, const T& qg_,
       const T& kg_) {
    const T& t = q.defined() ? q : k;
    if (!t.defined()) refuse("q or k is needed");
    if (t.dim() != 3) refuse("q and k must be (tokens, heads, d)");
    if (!t.is_cuda()) refuse("expected CUDA tensors");
    index = t.get_device();
    type = t.scalar_type();
    n = t.size(0);
    d = t.size(2);
    H_q = q.defined() ? q.size(1) : 0;
    H_k = 0;
    if (k.defined()) {
      if (k.dim() != 3 || k.size(0) != n || k.size(2) != d) refuse("q and k must share their tokens and head width");
      H_k = k.size(1);
    }
    B = 0;
    if (positions_.defined()) {
      if (cu_.defined() || pos0_.defined()) refuse("give positions or cu_seqlens (with pos0), not both");
      if (positions_.numel() != n) refuse("one position per token");
    } else if (cu_.defined()) {
      if (cu_.numel() < 1 || cu_.numel() > 0x7fffffff) refuse("cu_seqlens has B + 1 entries");
      B = (int32_t)(cu_.numel() - 1);
    }
    if (pos0_.defined() && (!cu_.defined() || pos0_.numel() != B)) refuse("pos0 is one start per cu_seqlens segment");
    if ((qg_.defined() && qg_.numel() != d) || (kg_.defined() && kg_.numel() != d))
      refuse("gammas must have d entries");
    if (H_q > 0x7fffffff || H_k > 0x7fffffff || d > 0x7fffffff ||
        (turns_.defined() && turns_.numel() > 0x3fffffff))
      refuse("sizes beyond 32 bits");
    cu = static_cast<const int32_t*>(flat(cu_, index, at::kInt, "cu_seqlens"));
    pos0 = static_cast<const int32_t*>(flat(pos0_, index, at::kInt, "pos0"));
    positions = static_cast<const int32_t*>(flat(positions_, index, at::kInt, "positions"));
    turns = static_cast<const uint64_t*>(flat(turns_, index, at::kLong, "turns"));
    rot = turns_.defined() ? (int32_t)(2 * turns_.numel()) : 0;
    qg = static_cast<const float*>(flat(qg_, index, at::kFloat, "q_gamma"));
    kg = static_cast<const float*>(flat(kg_, index, at::kFloat, "k_gamma"));
  }
};

// q, k, turns, cu_seqlens, positions, pos0, q_gamma, k_gamma, eps, interleaved, rot_scale, q_out, k_out, stream
PyObject* qk_norm_rope(PyObject* const* a, Py_ssize_t n) {
  arity(n, 14);
  const T &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
  const Rope r(q, k, tensor(a[2], "turns"), tensor(a[3], "cu_seqlens"), tensor(a[4], "positions"),
               tensor(a[5], "pos0"), tensor(a[6], "q_gamma"), tensor(a[7], "k_gamma"));
  const Tokens qt = tokens(q, r.index, r.type, "q"), kt = tokens(k, r.index, r.type, "k");
  const int32_t dt = dtype_of(r.type);
  Call call(r.index, a[13]);
  T q_out = tensor(a[11], "q_out"), k_out = tensor(a[12], "k_out");
  if (!q_out.defined() && q.defined()) q_out = like(q);
  if (!k_out.defined() && k.defined()) k_out = like(k);
  if (!same_shape(q, q_out) || !same_shape(k, k_out)) refuse("outputs must have their inputs' shapes");
  const Tokens qo = tokens(q_out, r.index, r.type, "q_out"), ko = tokens(k_out, r.index, r.type, "k_out");
  const int st = unlocked(f_rope, (nt_dtype)dt, qt.p, qt.stride, kt.p, kt.stride, r.n, (int32_t)r.H_q, (int32_t)r.H_k,
                        (int32_t)r.d, r.qg, r.kg, (float)number(a[8]), r.cu, r.B, r.pos0, r.positions, r.turns, r.rot,
                        flag(a[9]), (float)number(a[10]), qo.p, qo.stride, ko.p, ko.stride, call.stream);
  return result(st, {&q_out, &k_out});
}

// dq_out, dk_out, turns, q, k, cu_seqlens, positions, pos0, q_gamma, k_gamma, eps, interleaved, rot_scale, workspace,
// stream
PyObject* qk_norm_rope_bwd(PyObject* const* a, Py_ssize_t n) {
  arity(n, 15);
  const T &uq = tensor(a[0], "dq_out"), &uk = tensor(a[1], "dk_out"), &q = tensor(a[3], "q"), &k = tensor(a[4], "k"),
          &qg = tensor(a[8], "q_gamma"), &kg = tensor(a[9], "k_gamma");
  const Rope r(uq, uk, tensor(a[2], "turns"), tensor(a[5], "cu_seqlens"), tensor(a[6], "positions"),
               tensor(a[7], "pos0"), qg, kg);
  if (qg.defined() && (!q.defined() || !uq.defined() || q.sizes() != uq.sizes()))
    refuse("q's norm needs q and its upstream gradient, of one shape");
  if (kg.defined() && (!k.defined() || !uk.defined() || k.sizes() != uk.sizes()))
    refuse("k's norm needs k and its upstream gradient, of one shape");
  const Tokens uqt = tokens(uq, r.index, r.type, "dq_out"), ukt = tokens(uk, r.index, r.type, "dk_out");
  const Tokens qt = qg.defined() ? tokens(q, r.index, r.type, "q") : Tokens{};
  const Tokens kt = kg.defined() ? tokens(k, r.index, r.type, "k") : Tokens{};
  const int32_t dt = dtype_of(r.type);
  Call call(r.index, a[14]);
  T dq, dk, dqg, dkg, ws = tensor(a[13], "workspace");
  if (uq.defined()) dq = like(uq);
  if (uk.defined()) dk = like(uk);
  if (qg.defined()) dqg = like(qg);
  if (kg.defined()) dkg = like(kg);
  if (ws.defined()) {
    on_device(ws, r.index, "workspace");
    if (!ws.is_contiguous()) refuse("workspace must be contiguous");
  } else if (qg.defined() || kg.defined()) {
    ws = bytes(f_rope_bwd_ws((int32_t)r.d), uq.defined() ? uq : uk);
  }
  const int st = unlocked(f_rope_bwd, (nt_dtype)dt, uqt.p, uqt.stride, ukt.p, ukt.stride, qt.p, qt.stride, kt.p, kt.stride, r.n,
                            (int32_t)r.H_q, (int32_t)r.H_k, (int32_t)r.d, r.qg, r.kg, (float)number(a[10]), r.cu, r.B,
                            r.pos0, r.positions, r.turns, r.rot, flag(a[11]), (float)number(a[12]),
                            data(dq), r.H_q * r.d, data(dk), r.H_k * r.d, static_cast<float*>(data(dqg)),
                            static_cast<float*>(data(dkg)), data(ws), ws.defined() ? ws.nbytes() : 0, call.stream);
  return result(st, {&dq, &dk, &dqg, &dkg});
}

// The pages: address of the host struct, and their device.
struct Pages {
  const nt_kv_pages* p;
  int index;
  at::ScalarType type;
  Pages(PyObject* address, PyObject* device) {
    p = static_cast<const nt_kv_pages*>(PyLong_AsVoidPtr(address));
    if (!p) refuse("pages is needed");
    index = (int)integer(device);
    type = p->dtype == NT_BF16 ? at::kBFloat16 : at::kFloat;
  }
};
const int32_t* block_table(const T& t, int64_t B, int index, int32_t& max_pages) {
  if (t.dim() != 2 || t.size(0) != B || t.size(1) > 0x7fffffff)
    refuse("block_table must be (B = " + std::to_string(B) + ", max_pages)");
  max_pages = (int32_t)t.size(1);
  return static_cast<const int32_t*>(flat(t, index, at::kInt, "block_table"));
}

// pages, device, k, v, cu_seqlens, block_table, pos0, stream
PyObject* paged_write(PyObject* const* a, Py_ssize_t n) {
  arity(n, 8);
  const Pages g(a[0], a[1]);
  const T &k = need(a[2], "k"), &v = need(a[3], "v"), &cu = need(a[4], "cu_seqlens"), &pos0 = tensor(a[6], "pos0");
  if (k.dim() != 3 || k.sizes() != v.sizes() || k.size(1) != g.p->H_kv || k.size(2) != g.p->d)
    refuse("k and v must be (T, H_kv, d) of the pages");
  if (cu.numel() < 1 || cu.numel() > 0x7fffffff) refuse("cu_seqlens has B + 1 entries");
  const int32_t B = (int32_t)(cu.numel() - 1);
  if (pos0.defined() && pos0.numel() != B) refuse("pos0 is one start per cu_seqlens segment");
  const Tokens kt = tokens(k, g.index, g.type, "k"), vt = tokens(v, g.index, g.type, "v");
  int32_t max_pages;
  const int32_t* table = block_table(need(a[5], "block_table"), B, g.index, max_pages);
  const void *c = flat(cu, g.index, at::kInt, "cu_seqlens"), *p0 = flat(pos0, g.index, at::kInt, "pos0");
  Call call(g.index, a[7]);
  const int st = unlocked(f_write, g.p, kt.p, kt.stride, vt.p, vt.stride, k.size(0), static_cast<const int32_t*>(c), B,
                         static_cast<const int32_t*>(p0), table, max_pages, call.stream);
  return result(st, {});
}

// pages, device, src, dst, stream
PyObject* paged_copy(PyObject* const* a, Py_ssize_t n) {
  arity(n, 5);
  const Pages g(a[0], a[1]);
  const T &src = need(a[2], "src"), &dst = need(a[3], "dst");
  if (!src.is_cpu() || !dst.is_cpu()) refuse("src and dst are host tensors");
  if (src.scalar_type() != at::kInt || dst.scalar_type() != at::kInt || src.dim() != 1 || src.sizes() != dst.sizes())
    refuse("src and dst must be int32, one entry per copy");
  if (!src.is_contiguous() || !dst.is_contiguous()) refuse("src and dst must be contiguous");
  Call call(g.index, a[4]);
  const int st = unlocked(f_copy, g.p, static_cast<const int32_t*>(src.data_ptr()), static_cast<const int32_t*>(dst.data_ptr()),
                        src.numel(), call.stream);
  return result(st, {});
}

// pages, device, q, block_table, lengths, scale, out, lse, want_lse, workspace, stream
PyObject* paged_attn(PyObject* const* a, Py_ssize_t n) {
  arity(n, 11);
  const Pages g(a[0], a[1]);
  const int32_t d = g.p->d;
  const T &q = need(a[2], "q"), &lengths = need(a[4], "lengths");
  if (q.dim() != 3 || q.size(2) != d) refuse("q must be (B, H, d) with the pages' d");
  const int64_t B = q.size(0), H = q.size(1);
  if (B > 0x7fffffff || H > 0x7fffffff) refuse("sizes beyond 32 bits");
  if (lengths.numel() != B) refuse("one length per sequence");
  const Tokens qt = tokens(q, g.index, g.type, "q");
  int32_t max_pages;
  const int32_t* table = block_table(need(a[3], "block_table"), B, g.index, max_pages);
  const void* len = flat(lengths, g.index, at::kInt, "lengths");
  Call call(g.index, a[10]);
  T out = tensor(a[6], "out"), lse = tensor(a[7], "lse"), ws = tensor(a[9], "workspace");
  if (!out.defined()) out = like(q);
  else if (out.sizes() != q.sizes()) refuse("out must have q's shape");
  if (!lse.defined() && flag(a[8])) lse = fresh({H, B}, at::kFloat, g.index);
  if (lse.defined() && (lse.dim() != 2 || lse.size(0) != H || lse.size(1) != B)) refuse("lse must be (H, B)");
  if (ws.defined()) {
    on_device(ws, g.index, "workspace");
    if (!ws.is_contiguous()) refuse("workspace must be contiguous");
  } else {
    ws = bytes(f_attn_ws((int32_t)H, g.p->H_kv, d), q);
  }
  const float scale = a[5] == Py_None ? 1.0f / std::sqrt((float)d) : (float)number(a[5]);
  const int st = unlocked(f_attn, g.p, qt.p, qt.stride, (int32_t)B, (int32_t)H, table, max_pages,
                        static_cast<const int32_t*>(len), scale, flat(out, g.index, g.type, "out"),
                        static_cast<float*>(flat(lse, g.index, at::kFloat, "lse")), data(ws), ws.nbytes(),
                        call.stream);
  return result(st, {&out, &lse});
}

int32_t* ints(const T& t, int index, const char* name) { return static_cast<int32_t*>(flat(t, index, at::kInt, name)); }
int32_t int32_of(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < -0x80000000LL || v > 0x7fffffffLL) refuse(std::string(name) + " beyond 32 bits");
  return (int32_t)v;
}
int32_t segments(const T& cu, const char* name) {
  if (cu.numel() < 1 || cu.numel() > 0x7fffffff) refuse(std::string(name) + " has B + 1 entries");
  return (int32_t)(cu.numel() - 1);
}

// pages, device, k, v, slots, stream
PyObject* paged_write_slots(PyObject* const* a, Py_ssize_t n) {
  arity(n, 6);
  const Pages g(a[0], a[1]);
  const T &k = need(a[2], "k"), &v = need(a[3], "v"), &slots = need(a[4], "slots");
  if (k.dim() != 3 || k.sizes() != v.sizes() || k.size(1) != g.p->H_kv || k.size(2) != g.p->d)
    refuse("k and v must be (T, H_kv, d) of the pages");
  if (slots.numel() != k.size(0)) refuse("one slot per token");
  const Tokens kt = tokens(k, g.index, g.type, "k"), vt = tokens(v, g.index, g.type, "v");
  const void* s = flat(slots, g.index, at::kLong, "slots");
  Call call(g.index, a[5]);
  const int st = unlocked(f_write_slots, g.p, kt.p, kt.stride, vt.p, vt.stride, k.size(0),
                          static_cast<const int64_t*>(s), call.stream);
  return result(st, {});
}

// block_table, lengths, free_pages, n_free, page_size, new_lengths, tokens, stream
PyObject* paged_resize(PyObject* const* a, Py_ssize_t n) {
  arity(n, 8);
  const T &table = need(a[0], "block_table"), &lengths = need(a[1], "lengths"), &free_pages = need(a[2], "free_pages"),
          &n_free = need(a[3], "n_free"), &now = need(a[5], "new_lengths");
  if (!table.is_cuda()) refuse("expected CUDA tensors");
  const int index = table.get_device();
  const int64_t B = lengths.numel(), tokens = integer(a[6]);
  if (B > 0x7ffffffe || free_pages.numel() > 0x7fffffff) refuse("sizes beyond 32 bits");
  if (now.numel() != B) refuse("one new length per row");
  if (n_free.numel() != 1) refuse("n_free has one entry");
  if (tokens < 0) refuse("tokens must be >= 0");
  int32_t max_pages;
  int32_t* t = const_cast<int32_t*>(block_table(table, B, index, max_pages));
  int32_t *len = ints(lengths, index, "lengths"), *f = ints(free_pages, index, "free_pages"),
          *nf = ints(n_free, index, "n_free"), *nl = ints(now, index, "new_lengths");
  const int32_t page_size = int32_of(a[4], "page_size");
  Call call(index, a[7]);
  // one allocation for the four outputs, each a tensor over its part of it
  const int64_t ints_at = 8 * tokens;
  const T all = fresh({ints_at + 4 * (2 * B + 3)}, at::kByte, index);
  const T slots = part(all, 0, {tokens}, at::kLong), cu = part(all, ints_at, {B + 1}, at::kInt),
          pos0 = part(all, ints_at + 4 * (B + 1), {B}, at::kInt), lacking = part(all, ints_at + 4 * (2 * B + 1), {2}, at::kInt);
  const int st = unlocked(f_resize, nl, (int32_t)B, page_size, t, max_pages, len, f, (int32_t)free_pages.numel(), nf,
                          static_cast<int32_t*>(data(cu)), static_cast<int32_t*>(data(pos0)),
                          static_cast<int64_t*>(data(slots)), tokens, static_cast<int32_t*>(data(lacking)), call.stream);
  return result(st, {&cu, &pos0, &slots, &lacking});
}

// parents, cu_seqlens, max_new, pos0, bits, positions, stream
PyObject* draft_tree(PyObject* const* a, Py_ssize_t n) {
  arity(n, 7);
  const T &parents = need(a[0], "parents"), &cu = need(a[1], "cu_seqlens"), &pos0 = tensor(a[3], "pos0");
  if (!parents.is_cuda()) refuse("expected CUDA tensors");
  if (parents.dim() != 1) refuse("parents must be (tokens)");
  const int index = parents.get_device();
  const int64_t tokens = parents.numel();
  const int32_t B = segments(cu, "cu_seqlens"), max_new = int32_of(a[2], "max_new");
  if (pos0.defined() && pos0.numel() != B) refuse("pos0 is one start per cu_seqlens segment");
  const int32_t *p = ints(parents, index, "parents"), *c = ints(cu, index, "cu_seqlens"), *p0 = ints(pos0, index, "pos0");
  Call call(index, a[6]);
  T bits = tensor(a[4], "bits"), positions = tensor(a[5], "positions");
  const int64_t words = ((int64_t)max_new + 63) / 64;
  if (!bits.defined() && !positions.defined() && words > 0) {        // one allocation for both
    const T all = fresh({tokens * (8 * words + 4)}, at::kByte, index);
    bits = part(all, 0, {tokens, words}, at::kLong);
    positions = part(all, tokens * 8 * words, {tokens}, at::kInt);
  }
  if (!bits.defined()) bits = fresh({tokens, std::max<int64_t>(words, 0)}, at::kLong, index);
  else if (bits.dim() != 2 || bits.size(0) != tokens || bits.size(1) != words)
    refuse("bits must be (tokens, ceil(max_new / 64))");
  if (!positions.defined()) positions = fresh({tokens}, at::kInt, index);
  else if (positions.numel() != tokens) refuse("one position per token");
  const int st = unlocked(f_tree, p, c, B, tokens, max_new, p0, static_cast<int64_t*>(flat(bits, index, at::kLong, "bits")),
                          ints(positions, index, "positions"), call.stream);
  return result(st, {&bits, &positions});
}

// pages, device, kept, cu_kept, block_table, pos0, stream
PyObject* paged_keep(PyObject* const* a, Py_ssize_t n) {
  arity(n, 7);
  const Pages g(a[0], a[1]);
  const T &kept = need(a[2], "kept"), &cu = need(a[3], "cu_kept"), &pos0 = need(a[5], "pos0");
  const int32_t B = segments(cu, "cu_kept");
  if (pos0.numel() != B) refuse("pos0 is one start per cu_kept segment");
  int32_t max_pages;
  const int32_t* table = block_table(need(a[4], "block_table"), B, g.index, max_pages);
  const int32_t *k = ints(kept, g.index, "kept"), *c = ints(cu, g.index, "cu_kept"), *p0 = ints(pos0, g.index, "pos0");
  Call call(g.index, a[6]);
  const int st = unlocked(f_keep, g.p, k, kept.numel(), c, B, table, max_pages, p0, call.stream);
  return result(st, {});
}

// pages, device, q, cu_seqlens, block_table, lengths, max_new, bits, scale, out, lse, want_lse, workspace, stream
PyObject* paged_tree_attn(PyObject* const* a, Py_ssize_t n) {
  arity(n, 14);
  const Pages g(a[0], a[1]);
  const int32_t d = g.p->d;
  const T &q = need(a[2], "q"), &cu = need(a[3], "cu_seqlens"), &lengths = need(a[5], "lengths"), &bits = tensor(a[7], "bits");
  if (q.dim() != 3 || q.size(2) != d) refuse("q must be (tokens, H, d) with the pages' d");
  const int64_t tokens_ = q.size(0), H = q.size(1);
  if (H > 0x7fffffff) refuse("sizes beyond 32 bits");
  const int32_t B = segments(cu, "cu_seqlens"), max_new = int32_of(a[6], "max_new");
  if (lengths.numel() != B) refuse("one length per sequence");
  if (bits.defined() && (bits.dim() != 2 || bits.size(0) != tokens_ || bits.size(1) != ((int64_t)max_new + 63) / 64))
    refuse("bits must be (tokens, ceil(max_new / 64))");
  const Tokens qt = tokens(q, g.index, g.type, "q");
  int32_t max_pages;
  const int32_t* table = block_table(need(a[4], "block_table"), B, g.index, max_pages);
  const int32_t *c = ints(cu, g.index, "cu_seqlens"), *len = ints(lengths, g.index, "lengths");
  const int64_t* mask = static_cast<const int64_t*>(flat(bits, g.index, at::kLong, "bits"));
  Call call(g.index, a[13]);
  T out = tensor(a[9], "out"), lse = tensor(a[10], "lse"), ws = tensor(a[12], "workspace");
  if (!out.defined()) out = like(q);
  else if (out.sizes() != q.sizes()) refuse("out must have q's shape");
  if (!lse.defined() && flag(a[11])) lse = fresh({H, tokens_}, at::kFloat, g.index);
  if (lse.defined() && (lse.dim() != 2 || lse.size(0) != H || lse.size(1) != tokens_)) refuse("lse must be (H, tokens)");
  if (ws.defined()) {
    on_device(ws, g.index, "workspace");
    if (!ws.is_contiguous()) refuse("workspace must be contiguous");
  } else {
    ws = bytes(f_tree_attn_ws((int32_t)H, g.p->H_kv, d, max_new), q);
  }
  const float scale = a[8] == Py_None ? 1.0f / std::sqrt((float)d) : (float)number(a[8]);
  const int st = unlocked(f_tree_attn, g.p, qt.p, qt.stride, tokens_, (int32_t)H, c, B, max_new, table, max_pages, len,
                          mask, scale, flat(out, g.index, g.type, "out"),
                          static_cast<float*>(flat(lse, g.index, at::kFloat, "lse")), data(ws), ws.nbytes(),
                          call.stream);
  return result(st, {&out, &lse});
}

// Addresses of the C functions, in this order.
PyObject* bind(PyObject* const* a, Py_ssize_t n) {
  constexpr int kFunctions = 13;
  arity(n, kFunctions);
  void* p[kFunctions];
  for (int i = 0; i < kFunctions; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) refuse("a function's address is needed");
  }
  f_rope = reinterpret_cast<decltype(f_rope)>(p[0]);
  f_rope_bwd = reinterpret_cast<decltype(f_rope_bwd)>(p[1]);
  f_rope_bwd_ws = reinterpret_cast<decltype(f_rope_bwd_ws)>(p[2]);
  f_write = reinterpret_cast<decltype(f_write)>(p[3]);
  f_copy = reinterpret_cast<decltype(f_copy)>(p[4]);
  f_attn = reinterpret_cast<decltype(f_attn)>(p[5]);
  f_attn_ws = reinterpret_cast<decltype(f_attn_ws)>(p[6]);
  f_write_slots = reinterpret_cast<decltype(f_write_slots)>(p[7]);
  f_resize = reinterpret_cast<decltype(f_resize)>(p[8]);
  f_tree = reinterpret_cast<decltype(f_tree)>(p[9]);
  f_keep = reinterpret_cast<decltype(f_keep)>(p[10]);
  f_tree_attn = reinterpret_cast<decltype(f_tree_attn)>(p[11]);
  f_tree_attn_ws = reinterpret_cast<decltype(f_tree_attn_ws)>(p[12]);
  Py_RETURN_NONE;
}

// C++ exceptions end here: a mismatch as ValueError, torch's own as torch
// raises them.
template <PyObject* (*kFn)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return kFn(args, n);
  } catch (const Mismatch& m) {
    PyErr_SetString(PyExc_ValueError, m.text.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}
template <PyObject* (*kFn)(PyObject* const*, Py_ssize_t)>
constexpr PyCFunction method() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<kFn>));
}

PyMethodDef kMethods[] = {
    {"bind", method<bind>(), METH_FASTCALL, nullptr},
    {"qk_norm_rope", method<qk_norm_rope>(), METH_FASTCALL, nullptr},
    {"qk_norm_rope_bwd", method<qk_norm_rope_bwd>(), METH_FASTCALL, nullptr},
    {"paged_write", method<paged_write>(), METH_FASTCALL, nullptr},
    {"paged_copy", method<paged_copy>(), METH_FASTCALL, nullptr},
    {"paged_attn", method<paged_attn>(), METH_FASTCALL, nullptr},
    {"paged_write_slots", method<paged_write_slots>(), METH_FASTCALL, nullptr},
    {"paged_resize", method<paged_resize>(), METH_FASTCALL, nullptr},
    {"draft_tree", method<draft_tree>(), METH_FASTCALL, nullptr},
    {"paged_keep", method<paged_keep>(), METH_FASTCALL, nullptr},
    {"paged_tree_attn", method<paged_tree_attn>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_nt_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__nt_binding() { return PyModule_Create(&kModule); }
