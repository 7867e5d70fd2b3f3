// kda_check.cpp -- the tensors of a call checked and turned into addresses in one go (the Python module
// `_check`).
//
// A call that serves single tokens runs for a few microseconds on the device, and a dozen tensors looked
// at from Python take longer than that.  A checker holds what a call expects of them -- types, and shapes
// in symbols that the first tensor to show one binds -- and returns the numbers the C ABI wants, or None
// where anything is different; the Python wrappers then look closer and say what it is.  It only reads
// metadata.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <memory>
#include <sstream>
#include <string>
#include <vector>

namespace {

struct Dim {
  int symbol;     // index of the symbol
  int64_t plus;   // the extent is the symbol plus this
};
struct Entry {
  char type;      // f float32, i int32, v float32 or bfloat16 (the main type), s the main type, g float32 or,
                  // beside a bfloat16 main type, bfloat16
  std::vector<Dim> dims;
};
struct Checker {
  std::vector<Entry> entries;
  std::vector<std::string> symbols;
};

const char* kName = "kda_checker";

Checker* checker_of(PyObject* o) { return static_cast<Checker*>(PyCapsule_GetPointer(o, kName)); }
void destroy(PyObject* o) { delete checker_of(o); }

// make("x v T,H,d; cu i B+1; final f B,H,d") -> checker
PyObject* make(PyObject*, PyObject* arg) {
  const char* text = PyUnicode_AsUTF8(arg);
  if (!text) return nullptr;
  auto c = std::make_unique<Checker>();
  std::stringstream all(text);
  std::string item;
  while (std::getline(all, item, ';')) {
    std::stringstream words(item);
    std::string name, type, dims, dim;
    words >> name >> type >> dims;
    Entry e{type.size() == 1 ? type[0] : ' ', {}};
    std::stringstream list(dims);
    while (std::getline(list, dim, ',')) {
      int64_t plus = 0;
      if (const size_t at = dim.find('+'); at != std::string::npos) {
        plus = std::stoll(dim.substr(at + 1));
        dim = dim.substr(0, at);
      }
      int s = 0;
      while (s < (int)c->symbols.size() && c->symbols[s] != dim) ++s;
      if (s == (int)c->symbols.size()) c->symbols.push_back(dim);
      e.dims.push_back({s, plus});
    }
    if (e.dims.empty() || std::string("fivsg").find(e.type) == std::string::npos) {
      PyErr_Format(PyExc_ValueError, "cannot read %s", item.c_str());
      return nullptr;
    }
    c->entries.push_back(std::move(e));
  }
  return PyCapsule_New(c.release(), kName, destroy);
}

// check(checker, tensor, ...) -> (device number, symbols ..., addresses ..., 1 for bfloat16 of each v and g),
// or None
PyObject* check(PyObject*, PyObject* const* args, Py_ssize_t count) {
  const Checker* c = count > 0 ? checker_of(args[0]) : nullptr;
  if (!c) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "check(checker, tensor, ...)");
    return nullptr;
  }
  constexpr int kMost = 24;
  const int n = (int)c->entries.size(), symbols = (int)c->symbols.size();
  if (count != n + 1 || n > kMost || symbols > kMost) {
    PyErr_SetString(PyExc_TypeError, "the checker is for another number of tensors");
    return nullptr;
  }
  int64_t bound[kMost], address[kMost];
  long types[kMost];
  int typed = 0, index = -1;
  c10::ScalarType main_type = at::kFloat;
  for (int s = 0; s < symbols; ++s) bound[s] = -1;
  try {
    for (int i = 0; i < n; ++i) {
      const Entry& e = c->entries[i];
      PyObject* o = args[i + 1];
      if (!THPVariable_Check(o)) Py_RETURN_NONE;
      const at::Tensor& t = THPVariable_Unpack(o);
      if (!t.is_cuda() || t.layout() != at::kStrided || t.dim() != (int64_t)e.dims.size() || !t.is_contiguous()) Py_RETURN_NONE;
      const int on = t.get_device();
      if (index < 0) index = on;
      if (on != index) Py_RETURN_NONE;
      const c10::ScalarType type = t.scalar_type();
      const bool either = type == at::kFloat || type == at::kBFloat16;
      bool right = false;
      switch (e.type) {
        case 'f': right = type == at::kFloat; break;
        case 'i': right = type == at::kInt; break;
        case 'v': right = either; main_type = type; break;
        case 's': right = type == main_type; break;
        case 'g': right = either && (type == at::kFloat || main_type == at::kBFloat16); break;
      }
      if (!right) Py_RETURN_NONE;
      if (e.type == 'v' || e.type == 'g') types[typed++] = type == at::kBFloat16;
      const auto sizes = t.sizes();
      for (size_t k = 0; k < e.dims.size(); ++k) {
        const int64_t extent = sizes[k] - e.dims[k].plus;
        int64_t& b = bound[e.dims[k].symbol];
        if (b < 0) b = extent;
        if (b != extent || extent < 0 || extent > INT32_MAX) Py_RETURN_NONE;  // (the C ABI's are 32 bits)
      }
      address[i] = reinterpret_cast<int64_t>(t.data_ptr());
    }
  } catch (const std::exception&) {
    Py_RETURN_NONE;
  }
  PyObject* r = PyTuple_New(1 + symbols + n + typed);
  if (!r) return nullptr;
  int at = 0;
  PyTuple_SET_ITEM(r, at++, PyLong_FromLong(index));
  for (int s = 0; s < symbols; ++s) PyTuple_SET_ITEM(r, at++, PyLong_FromLongLong(bound[s]));
  for (int i = 0; i < n; ++i) PyTuple_SET_ITEM(r, at++, PyLong_FromLongLong(address[i]));
  for (int k = 0; k < typed; ++k) PyTuple_SET_ITEM(r, at++, PyLong_FromLong(types[k]));
  return r;
}

PyMethodDef methods[] = {
    {"make", make, METH_O, "make(expectations) -> checker"},
    {"check", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(check)), METH_FASTCALL,
     "check(checker, tensor, ...) -> numbers for the C ABI, or None"},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_check", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__check(void) { return PyModule_Create(&module); }
