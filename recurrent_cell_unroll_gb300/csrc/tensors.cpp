// Lists of torch tensors as the table that rcu_adamw_step takes (include/rcu.h): the part
// of the Python binding that looks at hundreds of tensors a call, where each check costs
// some 50 ns from Python (1.4 us a tensor; 0.1 us here).  No computation and no CUDA call.
#include <cstdint>

#include <torch/csrc/autograd/python_variable.h>

#include "rcu.h"

namespace {

static_assert(sizeof(rcu_adamw_tensor) == 72, "binding.py makes room for 72 bytes a tensor");

const at::Tensor *tensor_of(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

int type_of(const at::Tensor &t) {
  return t.scalar_type() == at::kFloat ? RCU_F32 : t.scalar_type() == at::kBFloat16 ? RCU_BF16 : -1;
}
// n dense values on the device.
bool dense(const at::Tensor *t, int64_t device, int64_t n) {
  return t && t->is_cuda() && t->get_device() == device && t->layout() == at::kStrided && t->numel() == n &&
         t->is_contiguous();
}

// A state: fp32 values, or (codes, exponents) of 8 bits.
bool state(PyObject *o, int64_t device, int64_t n, void **values, int8_t **exps) {
  if (!PyTuple_Check(o)) {
    const at::Tensor *t = tensor_of(o);
    if (!dense(t, device, n) || t->scalar_type() != at::kFloat) return false;
    *values = t->data_ptr();
    return true;
  }
  if (PyTuple_GET_SIZE(o) != 2) return false;
  const at::Tensor *codes = tensor_of(PyTuple_GET_ITEM(o, 0)), *e = tensor_of(PyTuple_GET_ITEM(o, 1));
  const int64_t blocks = (n + RCU_STATE8_BLOCK - 1) / RCU_STATE8_BLOCK;
  if (!dense(codes, device, n) || codes->scalar_type() != at::kChar || !dense(e, device, blocks) ||
      e->scalar_type() != at::kChar)
    return false;
  *values = codes->data_ptr();
  *exps = static_cast<int8_t *>(e->data_ptr());
  return true;
}

bool row_of(PyObject *p, PyObject *g, PyObject *m, PyObject *v, PyObject *copy, int64_t device,
            rcu_adamw_tensor *row) {
  const at::Tensor *pt = tensor_of(p), *gt = tensor_of(g);
  if (!pt || !gt || !dense(pt, device, pt->numel()) || !dense(gt, device, pt->numel()) ||
      gt->sizes() != pt->sizes() || type_of(*pt) < 0 || type_of(*gt) < 0)
    return false;
  rcu_adamw_tensor r{};
  r.p = pt->data_ptr(), r.g = gt->data_ptr(), r.n = pt->numel();
  r.p_type = type_of(*pt), r.g_type = type_of(*gt);
  if (!state(m, device, r.n, &r.m, &r.m_exp) || !state(v, device, r.n, &r.v, &r.v_exp) ||
      PyTuple_Check(m) != PyTuple_Check(v))
    return false;
  if (copy != Py_None) {
    const at::Tensor *ct = tensor_of(copy);
    if (!dense(ct, device, r.n) || ct->scalar_type() != at::kBFloat16) return false;
    r.copy = ct->data_ptr();
  }
  *row = r;
  return true;
}

struct List {  // a list or tuple, held while it is read
  PyObject *o;
  explicit List(PyObject *from) : o(PySequence_Fast(from, "expected a list of tensors")) {}
  ~List() { Py_XDECREF(o); }
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(o); }
  PyObject *operator[](Py_ssize_t k) const { return PySequence_Fast_GET_ITEM(o, k); }
};

// adamw_rows(rows, params, grads, m, v, copies, device): fills the buffer `rows`, a row a
// tensor (of a gradient of None: zeros), and returns the number of the first tensor that
// does not fit, or -1.
PyObject *adamw_rows(PyObject *, PyObject *args) {
  Py_buffer room;
  PyObject *p, *g, *m, *v, *copies;
  long long device;
  if (!PyArg_ParseTuple(args, "w*OOOOOL", &room, &p, &g, &m, &v, &copies, &device)) return nullptr;
  PyObject *result = nullptr;
  try {
    const List ps(p), gs(g), ms(m), vs(v), cs(copies == Py_None ? p : copies);
    if (ps.o && gs.o && ms.o && vs.o && cs.o) {
      const Py_ssize_t count = ps.size();
      if (gs.size() != count || ms.size() != count || vs.size() != count || cs.size() != count ||
          room.len < (Py_ssize_t)(count * sizeof(rcu_adamw_tensor))) {
        PyErr_SetString(PyExc_ValueError, "params, grads, m, v and copies must be lists of one length");
      } else {
        auto *rows = static_cast<rcu_adamw_tensor *>(room.buf);
        Py_ssize_t k = 0;
        for (; k < count; ++k) {
          rows[k] = {};
          if (gs[k] == Py_None) continue;
          if (!row_of(ps[k], gs[k], ms[k], vs[k], copies == Py_None ? Py_None : cs[k], device, rows + k)) break;
        }
        result = PyLong_FromSsize_t(k < count ? k : -1);
      }
    }
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  PyBuffer_Release(&room);
  return result;
}

// changed(params, grads, copies): tells autograd of parameters and their copies (a list, or
// None) that have been changed in place: those that have a gradient.
PyObject *changed(PyObject *, PyObject *args) {
  PyObject *p, *g, *copies;
  if (!PyArg_ParseTuple(args, "OOO", &p, &g, &copies)) return nullptr;
  try {
    const List ps(p), gs(g), cs(copies == Py_None ? p : copies);
    if (!ps.o || !gs.o || !cs.o) return nullptr;
    auto tell = [](PyObject *o) {
      const at::Tensor *t = tensor_of(o);
      if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
    };
    for (Py_ssize_t k = 0; k < ps.size() && k < gs.size(); ++k) {
      if (gs[k] == Py_None) continue;
      tell(ps[k]);
      if (copies != Py_None && k < cs.size()) tell(cs[k]);
    }
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"adamw_rows", adamw_rows, METH_VARARGS, "The table of an AdamW step's tensors."},
                         {"changed", changed, METH_VARARGS, "Tensors that have been changed in place."},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "tensors", "Lists of tensors as the C ABI takes them.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_tensors() { return PyModule_Create(&module); }
