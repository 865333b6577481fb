// Argument marshalling for calls that take lists of tensors: their types, sizes and addresses into
// host arrays in one call (from Python each of these costs a tenth of a microsecond a tensor,
// more than the kernels of a small list).  Called with the interpreter's lock held (ctypes.PyDLL).
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <vector>

#include "scopt.h"

namespace {
// The tensor's type if it is one that the library takes: a contiguous float32 or bfloat16 tensor on `device`.
int type_of(const at::Tensor& t, int device) {
    if (t.layout() != at::kStrided || !t.is_cuda() || t.get_device() != device || !t.is_contiguous()) return -1;
    return t.scalar_type() == at::kFloat ? SC_F32 : t.scalar_type() == at::kBFloat16 ? SC_BF16 : -1;
}
}  // namespace

// Fills the arrays (`n` entries each) from a list; like: a list that types and sizes have to match, or
// NULL.  Returns -1, or the index of the first entry that is not as described.
extern "C" __attribute__((visibility("default"))) int scopt_tensor_table(PyObject* list, PyObject* like, int n, int device,
                                                                        int* dtypes, int64_t* sizes, void** where) {
    if (!PyList_Check(list) || PyList_GET_SIZE(list) != n) return 0;
    if (like && (!PyList_Check(like) || PyList_GET_SIZE(like) != n)) return 0;
    int i = 0;
    try {
        for (; i < n; ++i) {
            PyObject* item = PyList_GET_ITEM(list, i);
            if (!THPVariable_Check(item)) return i;
            const at::Tensor& t = THPVariable_Unpack(item);
            const int type = type_of(t, device);
            if (type < 0) return i;
            if (like) {
                const at::Tensor& u = THPVariable_Unpack(PyList_GET_ITEM(like, i));
                if (u.scalar_type() != t.scalar_type() || !u.sizes().equals(t.sizes())) return i;
            }
            dtypes[i] = type;
            sizes[i] = t.numel();
            where[i] = t.data_ptr();
        }
    } catch (...) {
        return i;
    }
    return -1;
}

// Whether tensors can be written while others are read: no two outputs share memory, and an output shares an
// input's only where it is that input (the same entry, from its start).  Returns -1, or the index of the first output
// found that is not so.
extern "C" __attribute__((visibility("default"))) int scopt_overlap(int n, const int* dtypes, const int64_t* sizes,
                                                                   void* const* in, void* const* out) {
    struct Range {
        uintptr_t from, to;
        int i;
    };
    try {
        auto range = [&](void* const* p, int i) {
            const uintptr_t from = (uintptr_t)p[i];
            return Range{from, from + (uintptr_t)sizes[i] * (dtypes[i] == SC_BF16 ? 2 : 4), i};
        };
        std::vector<Range> written;
        written.reserve(n);
        for (int i = 0; i < n; ++i)
            if (sizes[i] > 0) written.push_back(range(out, i));
        auto before = [](const Range& a, const Range& b) { return a.from < b.from; };
        if (!std::is_sorted(written.begin(), written.end(), before)) std::sort(written.begin(), written.end(), before);
        for (size_t k = 1; k < written.size(); ++k)
            if (written[k].from < written[k - 1].to) return written[k].i;
        if (in == out) return -1;
        for (int i = 0; i < n; ++i) {
            if (sizes[i] == 0) continue;
            const Range r = range(in, i);
            auto w = std::upper_bound(written.begin(), written.end(), r.from,
                                      [](uintptr_t at, const Range& x) { return at < x.to; });  // the first that ends behind
            for (; w != written.end() && w->from < r.to; ++w)
                if (w->i != i || w->from != r.from) return w->i;
        }
    } catch (...) {
        return 0;
    }
    return -1;
}
