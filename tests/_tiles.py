"""Shapes that take each of the tiles of the MXFP4 products, with the choice that is expected of the library: sizes that no
tile divides beside whole ones, one step of 128 k to forty, outputs whose rows allow 16-byte stores and those that do not."""
import ctypes

from block_quantized_matrix_amd import bqm

# (index of the tile, M, N, K): 256 x 256; 128 x 128 in one and two shares of K; 128 x 64 in two; 128 x 32 in four;
# 64 x 64 in four; 64 x 32 and 64 x 16 in eight; 32 x 16 in sixteen
DENSE = [(0, 145, 17453, 32), (0, 133, 18363, 288), (0, 700, 12820, 224), (0, 270, 21994, 544), (0, 2856, 2944, 1472),
         (0, 264, 21992, 2112), (0, 2481, 5353, 1600), (1, 129, 21821, 1696), (1, 66, 17299, 608), (1, 397, 9089, 1600),
         (2, 66, 17773, 1568), (2, 3270, 537, 1760), (2, 453, 5521, 3168), (2, 1974, 1302, 5024), (3, 35, 17011, 1440),
         (3, 834, 1591, 1600), (3, 38, 22858, 3168), (4, 1, 16882, 1056), (4, 7, 21989, 1536), (4, 8, 18525, 5088),
         (5, 34, 8458, 2112), (5, 374, 1081, 4192), (6, 805, 381, 2080), (6, 218, 1357, 3200), (6, 4400, 5, 3168),
         (7, 653, 208, 4192), (7, 129, 22, 2144), (8, 52, 38, 4160), (8, 481, 4, 5024)]

# (index of the tile, T, E, top_k, N, K): 64 x 16 in four shares of K; 256 x 128; 256 x 64; 128 x 64; 128 x 32
INDEXED = [(0, 1, 16, 4, 777, 1696), (0, 4, 40, 2, 516, 2176), (1, 300, 6, 2, 530, 1696), (1, 173, 3, 3, 1044, 544),
           (2, 101, 12, 2, 301, 1696), (2, 260, 16, 1, 516, 2112), (3, 47, 10, 2, 389, 1696), (3, 64, 16, 2, 644, 3104),
           (4, 33, 40, 4, 261, 1696), (4, 90, 60, 2, 516, 2112)]

# rows of a decode product, by the runs of eight that a workgroup takes: every count of row tiles, whole and half
DECODE = {1: 2041, 2: 4096, 3: 5125, 5: 8200, 6: 12285, 7: 12290, 8: 16380, 9: 16391, 10: 20480, 11: 21001, 13: 26621, 14: 26625,
          15: 30001, 16: 32761, 17: 34001}


def _fn(name, args, res=ctypes.c_int):
    f = getattr(bqm.lib(), name)
    f.argtypes, f.restype = args, res
    return f


def dense_choice(M, N, K):
    return _fn("bqm_internal_qmm_mxfp4_choice", [ctypes.c_int64] * 3)(M, N, K)


def indexed_choice(E, N, slots):
    return _fn("bqm_internal_qmm_id_mxfp4_choice", [ctypes.c_int, ctypes.c_int64, ctypes.c_int])(E, N, slots)


def decode_runs(N):
    return _fn("bqm_internal_qmv_mxfp4_runs", [ctypes.c_int64], ctypes.c_int64)(N)
