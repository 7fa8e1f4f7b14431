/* args.c -- the checks of a binding call's tensors in one native call: on the device, of the type, contiguous
 * and of the shape. In Python they were more than half of a block-tables call (7 of 13.5 us for its 16
 * tensors), on a decode step's critical path. A tensor is looked at through the exchange table of the
 * DLPack standard that torch publishes (torch.Tensor.__dlpack_c_exchange_api__).
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/dlpack.h>

#define MAX_TYPES 16

static const DLPackExchangeAPI *api;
static PyTypeObject *tensor_type;
static struct {
    PyObject *dtype;
    int code, bits;
} types[MAX_TYPES];
static int n_types;

/* setup(torch.Tensor, [(dtype, DLPack type code, bits), ...]) */
static PyObject *setup(PyObject *self, PyObject *args) {
    PyObject *type, *list;
    if (!PyArg_ParseTuple(args, "OO!", &type, &PyList_Type, &list)) return NULL;
    if (!PyType_Check(type)) return PyErr_Format(PyExc_TypeError, "a type is expected");
    if (PyList_GET_SIZE(list) > MAX_TYPES) return PyErr_Format(PyExc_ValueError, "too many types");
    PyObject *capsule = PyObject_GetAttrString(type, "__dlpack_c_exchange_api__");
    if (!capsule) return NULL;
    const DLPackExchangeAPI *a = PyCapsule_GetPointer(capsule, "dlpack_exchange_api");
    Py_DECREF(capsule);   /* (the table is static) */
    if (!a) return NULL;
    if (a->header.version.major != DLPACK_MAJOR_VERSION || !a->dltensor_from_py_object_no_sync)
        return PyErr_Format(PyExc_ImportError, "DLPack %u of torch is not the one of its headers", a->header.version.major);
    for (Py_ssize_t i = 0; i < PyList_GET_SIZE(list); i++) {
        PyObject *dtype;
        int code, bits;
        if (!PyArg_ParseTuple(PyList_GET_ITEM(list, i), "Oii", &dtype, &code, &bits)) return NULL;
        Py_INCREF(dtype);
        types[i].dtype = dtype;
        types[i].code = code;
        types[i].bits = bits;
    }
    n_types = (int)PyList_GET_SIZE(list);
    Py_INCREF(type);
    tensor_type = (PyTypeObject *)type;
    api = a;
    Py_RETURN_NONE;
}

static int fits(PyObject *t, PyObject *dtype, PyObject *shape, long device, DLTensor *d) {
    if (!PyObject_TypeCheck(t, tensor_type)) return 0;
    if (api->dltensor_from_py_object_no_sync(t, d) != 0) {
        PyErr_Clear();
        return 0;
    }
    if (d->device.device_type != kDLCUDA || d->device.device_id != device || d->dtype.lanes != 1) return 0;
    int i = 0;
    while (i < n_types && types[i].dtype != dtype) i++;
    if (i == n_types || types[i].code != d->dtype.code || types[i].bits != d->dtype.bits) return 0;
    int64_t step = 1;
    int empty = 0;
    for (int k = 0; k < d->ndim; k++) empty |= d->shape[k] == 0;
    for (int k = d->ndim - 1; k >= 0 && d->strides && !empty; k--) {
        if (d->shape[k] != 1 && d->strides[k] != step) return 0;
        step *= d->shape[k];
    }
    if (shape == Py_None) return 1;
    if (!PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != d->ndim) return 0;
    for (int k = 0; k < d->ndim; k++) {
        const long long n = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, k));
        if (n == -1 && PyErr_Occurred()) PyErr_Clear();
        if (n != d->shape[k]) return 0;
    }
    return 1;
}

/* take(device, tensors, dtypes, shapes): tuples of one length, of tensors or None, of their types and of their
 * shapes or None. A list of addresses (None for None), or None when a tensor is not as it should be. */
static PyObject *take(PyObject *self, PyObject *const *args, Py_ssize_t n_args) {
    if (n_args != 4 || !api || !PyTuple_Check(args[1]) || !PyTuple_Check(args[2]) || !PyTuple_Check(args[3]))
        return PyErr_Format(PyExc_TypeError, "take(device, tensors, dtypes, shapes) after setup()");
    const Py_ssize_t n = PyTuple_GET_SIZE(args[1]);
    if (PyTuple_GET_SIZE(args[2]) != n || PyTuple_GET_SIZE(args[3]) != n)
        return PyErr_Format(PyExc_TypeError, "tuples of one length are expected");
    const long device = PyLong_AsLong(args[0]);
    if (device == -1 && PyErr_Occurred()) return NULL;
    PyObject *out = PyList_New(n);
    if (!out) return NULL;
    for (Py_ssize_t i = 0; i < n; i++) {
        PyObject *t = PyTuple_GET_ITEM(args[1], i), *p = Py_None;
        DLTensor d;
        if (t == Py_None) {
            Py_INCREF(p);
        } else if (fits(t, PyTuple_GET_ITEM(args[2], i), PyTuple_GET_ITEM(args[3], i), device, &d)) {
            p = PyLong_FromVoidPtr(d.data ? (char *)d.data + d.byte_offset : NULL);
            if (!p) {
                Py_DECREF(out);
                return NULL;
            }
        } else {
            Py_DECREF(out);
            Py_RETURN_NONE;
        }
        PyList_SET_ITEM(out, i, p);
    }
    return out;
}

static PyMethodDef methods[] = {{"setup", setup, METH_VARARGS, NULL},
                                {"take", (PyCFunction)(void (*)(void))take, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_args", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__args(void) { return PyModule_Create(&module); }
