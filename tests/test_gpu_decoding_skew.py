"""Insertion where one list is far longer than the others, so that the launch,
which goes by the mean, gives it one CTA a head and more candidates than that
keeps in registers."""
import pytest

from test_gpu_decoding import run_insert

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B,at,long,cap,Hkv", [(64, 0, 16384, 300, 2), (64, 31, 11000, 300, 2), (100, 99, 10300, 64, 1),
                                              (40, 7, 20000, 150, 9), (3, 1, 24000, 2000, 1)])
def test_one_long_list_among_short(B, at, long, cap, Hkv, in_place):
    ms = [long if b == at else b % 3 for b in range(B)]
    run_insert([cap - b % 2 for b in range(B)], ms, cap, Hkv, cap // 8, B + Hkv, d=8, in_place=in_place)
