"""Rings whose last tile begins less than a tile before position 2^31: what
lies behind the query's row in that tile has no positions, and no influence."""
import pytest
import torch

from orthogonal_reparameterized_02_amd import poetx as P
from gpu_util import to_f64
from oracle import long_context_oracle as L
from test_gpu_kv4 import close, run, setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    P.lib()


TOP = 2 ** 31 - 1


def reference(st):
    """The same rows at positions that a host array can hold; the sinks so far
    away that a bias hides them there too (slopes are 2^-4 and more)."""
    c, R = st["c"], st["c"]["rows"] - st["c"]["s"]
    lens = [c["s"] + (n - c["s"]) % R + 64 * R for n in c["len"]]
    return L.window_decode(to_f64(st["q"]), to_f64(st["k"]), to_f64(st["v"]), lens, c["w"], c["s"], True, None, 0.0,
                           None if st["slopes"] is None else to_f64(st["slopes"]))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("rows,window,sinks", [(192, 33, 2), (192, 35, 0), (256, 97, 4), (192, 1, 0), (64, 62, 2)])
def test_the_last_positions(rows, window, sinks, bias, four, dt):
    st = setup(dict(len=[TOP, TOP - 1, TOP - 3, TOP - 20, TOP - 31, TOP - 32, TOP // 2], rows=rows, Hq=4, Hkv=2, D=64, w=window, s=sinks,
                    ring=True, bias=bias), dt, four)
    close("o", run(st, four), reference(st), dt)
