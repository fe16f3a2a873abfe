"""The shapes of tests/test_gpu_mxfp4_tiles.py take every tile of the MXFP4 products.  No GPU needed."""
from tests import _tiles


def test_dense_shapes_take_every_tile():
    for tile, M, N, K in _tiles.DENSE:
        assert _tiles.dense_choice(M, N, K) == tile, (M, N, K)
    for tile in range(9):
        mine = [s for s in _tiles.DENSE if s[0] == tile]
        assert any(N % 4 for _, _, N, _ in mine) and any(M % 16 for _, M, _, _ in mine)
        assert max(-(-K // 128) for *_, K in mine) > 12  # past one turn of the stages
    assert _tiles.dense_choice(1 << 30, 1 << 30, 64) == -1


def test_indexed_shapes_take_every_tile():
    for tile, T, E, top_k, N, K in _tiles.INDEXED:
        assert _tiles.indexed_choice(E, N, T * top_k) == tile, (T, E, top_k, N)
    assert {s[0] for s in _tiles.INDEXED} == set(range(5))


def test_decode_rows_take_every_count_of_tiles():
    for runs, N in _tiles.DECODE.items():
        assert _tiles.decode_runs(N) == runs, N
    assert {(r + 1) // 2 for r in _tiles.DECODE} == set(range(1, 10))
    assert max(_tiles.decode_runs(n) for n in range(1, 200000, 7)) == 17
