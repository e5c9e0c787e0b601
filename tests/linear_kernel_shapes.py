"""Products that reach each kernel behind logra_linear and its gradients, with ragged edges:
C [M x N] with K terms, so (T, d, k) of the forward product, (T, k, d) of the input's
gradient and (d, k, T) of the weight's.  test_launches_step.py holds each to its kernel, on
the CPU; test_gpu_linear_kernels.py to its results.
"""
from collections import namedtuple

Shape = namedtuple("Shape", "kernel once split M N K")
# kernel: few (up to 16 rows, forward only), or rows x columns of the tile; once: one tile
# of rows, whose columns are read by nobody else; split: pieces of K, joined by a second launch
SHAPES = [
    Shape("few", False, False, 13, 517, 1003),
    Shape("64x64", True, False, 19, 205, 71),
    Shape("64x64", True, True, 63, 403, 1101),
    Shape("64x64", False, False, 301, 1003, 75),
    Shape("64x64", False, True, 130, 203, 2051),
    Shape("64x128", True, False, 41, 20001, 73),
    Shape("64x128", True, False, 61, 60001, 520),
    Shape("64x128", True, True, 23, 12005, 8195),
    Shape("64x128", False, False, 200, 8953, 1537),
    Shape("64x128", False, True, 201, 1027, 2053),
    Shape("256x128", False, False, 803, 5003, 43),
    Shape("256x128", False, False, 2047, 4090, 4101),
    Shape("256x128", False, True, 131, 4091, 8203),
    Shape("256x256", False, False, 401, 20003, 61),
    Shape("256x256", False, False, 8190, 4090, 1101),
    Shape("256x256", False, True, 1301, 2501, 8203),
]

# Activation gradients with a bias gradient: rows, columns, and whether strips of 256 columns
# (else 16) are added up, and in how many chunks of rows.
BIAS_SHAPES = [
    (1024, 777, False, 1), (1, 10240, False, 1), (1023, 10239, False, 1),
    (1025, 777, True, 129), (2050, 4099, True, 52), (5000, 10249, True, 25), (40, 10249, True, 5),
    (9, 10241, True, 2), (8, 10241, True, 1), (1, 70001, True, 1), (4100, 36, True, 513),
    (8200, 257, True, 342), (130, 300001, True, 1),
]
FORMS = ("forward", "input", "weight")


def form_of(shape, form):
    """(T, d, k) of the product in one of its forms."""
    M, N, K = shape[3:]
    return {"forward": (M, N, K), "input": (M, K, N), "weight": (K, M, N)}[form]


def has(shape, form):
    return form == "forward" or shape.kernel != "few"
