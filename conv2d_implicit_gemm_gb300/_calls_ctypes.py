"""The per-token calls through ctypes: what the package uses where the extension
module _calls has not been built or does not fit the interpreter.  The same
functions with the same checks; converting the 30 arguments of an attention call
takes 6.6 us here and 0.2 us there (on an x86 host).
"""

import ctypes
import operator
import types

# one letter an argument: p pointer, l long long, i int, f float, b bytes
KINDS = {"oidnx_linear": "plplpplpliiiiip",
         "oidnx_qk_norm_rope": "pllpllpllpllpllpllppfpplppliiiiiiip",
         "oidnx_window_attention": "plllplllplllplllpppiiiiiiiifip",
         "oidnx_block_norm": "plplplplippippfpliplplpiiffiiiip",
         "oidnx_qk_norm_rope_axes": "pllpllpllpllpllpllippfpplplibpliiiiiiip",
         "oidnx_cross_attention": "plllplllplllplllppppliiiiiifip"}
_TYPES = {"p": ctypes.c_void_p, "b": ctypes.c_char_p, "l": ctypes.c_longlong, "i": ctypes.c_int, "f": ctypes.c_float}
_RANGE = {"p": (0, 2 ** 64 - 1), "l": (-2 ** 63, 2 ** 63 - 1), "i": (-2 ** 31, 2 ** 31 - 1)}


def _convert(name, kinds, args):
    if len(args) != len(kinds):
        raise TypeError(f"{name} takes {len(kinds)} arguments ({len(args)} given)")
    out = []
    for n, (kind, a) in enumerate(zip(kinds, args)):
        if kind == "f":
            out.append(float(a))
        elif kind in "pb" and a is None:
            out.append(None)
        elif kind == "b":
            if not isinstance(a, bytes):
                raise TypeError(f"{name}: argument {n + 1} is no bytes object")
            out.append(a)
        else:
            v, (low, high) = operator.index(a), _RANGE[kind]
            if not low <= v <= high:
                raise OverflowError(f"{name}: argument {n + 1} is beyond its C type")
            out.append(v)
    return out


def bind(lib):
    """The calls of the loaded library, each by position and returning the status."""
    calls = types.SimpleNamespace()
    for name, kinds in KINDS.items():
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = [_TYPES[k] for k in kinds]

        def call(*args, _fn=fn, _name=name, _kinds=kinds):
            return _fn(*_convert(_name, _kinds, args))

        setattr(calls, name, call)
    return calls
