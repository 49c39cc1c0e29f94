"""What the packed cache's binding refuses before a call is made, on descriptions of tensors (no GPU)."""
import pytest

torch = pytest.importorskip("torch")

from decode_megakernel_persistent_gb300 import build as llbuild
from decode_megakernel_persistent_gb300 import ll
from test_kvq_host import _Fake, fake_cache


@pytest.fixture(scope="module", autouse=True)
def _lib():
    llbuild.build()


def test_read_into_one_tensor():
    """Two threads would write each element, in no order."""
    c, rows, lens = fake_cache(), _Fake((2, 3, 2, 64), torch.bfloat16, "cuda:0"), _Fake((2,), torch.int32, "cuda:0")
    with pytest.raises(ll.LLError, match="same rows"):
        ll.ll_kvq_read(c, rows, rows, lens)
    with pytest.raises(ll.LLError, match="same rows"):
        c.read(rows, rows, lens, lens)
