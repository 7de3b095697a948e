"""Attention of long prompts over their own keys and behind others', against the
definition in 64 bits with the tolerances of the other tests of attention."""
import pytest

from gpu_util import note
from test_gpu_kv_attend import BF, F8, HF, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name,a", [
    ("own keys", (BF, BF, 4, 2, 64, 16, [1500, 1100, 7], [1500, 1100, 7])),
    ("behind keys of its own", (HF, HF, 5, 1, 128, 16, [2300, 1300], [1201, 1])),
    ("one byte", (HF, F8, 2, 1, 64, 64, [1409], [1409])),
    ("behind shared keys", (BF, BF, 4, 1, 128, 16, [1700, 1610, 640], [1060, 970, 1], [0, 3], [624])),
    ("head size 256", (BF, BF, 2, 1, 256, 16, [1100], [1030])),
])
def test_long_prompts(name, a):
    note(f"kv attend prompts {name}")
    Case(*a).test()
