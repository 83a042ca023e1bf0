"""Which kernels mxq_linear_ce_* take for sizes, from the tests' build of the library (not a test module)."""
import ctypes as C
import functools

NAMES = {(256, 256, 2): "Many", (128, 256, 3): "Half", (128, 128, 4): "Deep", (128, 128, 2): "Twin", (128, 32, 3): "Few",
         (64, 64, 4): "Small", (64, 32, 6): "Slim", (128, 128, 1): "Outer"}
LOGITS = ("Slim", "Few", "Small", "Deep", "Twin", "Half", "Many")
OF = {"forward": LOGITS, "dz": LOGITS, "dx": ("Few", "Twin", "Deep", "Many"), "dw": ("Outer", "Deep", "Twin", "Many")}
SHIPPED, LOOP = 1 << 27, 1    # logits of a piece: in the library, in the tests' build


@functools.cache
def _fn():
    from fp4_microscaling_quantization_amd import build
    fn = C.CDLL(build.LOOP_LIB).mxq_linear_ce_kernels
    fn.argtypes, fn.restype = [C.c_int64] * 4 + [C.c_void_p] * 2, None
    return fn


def kernels(rows, hidden, vocab, piece=SHIPPED):
    """{"forward", "dz", "dx", "dw": (tile, whether a last step may be cut), "pieces", "width", "slabs"}"""
    tiles, plan = (C.c_int32 * 16)(), (C.c_int32 * 3)()
    _fn()(rows, hidden, vocab, piece, tiles, plan)
    got = {name: (NAMES[tuple(tiles[4 * i:4 * i + 3])], bool(tiles[4 * i + 3])) for i, name in enumerate(OF)}
    return {**got, "pieces": plan[0], "width": plan[1], "slabs": plan[2]}
