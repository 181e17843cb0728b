"""GPU checks of commits whose launches need shared memory around what a kernel has without asking for more, in processes that
asked for none before."""
import subprocess
import sys

import pytest

from tests import _drafts as R

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def commit_of(B, H, M, dk, dv, dtype, with_path):
    """One linear commit of M tokens for every sequence, the first and the last head against 64 bits."""
    from log_linear_attention_gb300 import binding as lla
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(M + dk)
    k, v = (torch.randn(B, H, M, d, device="cuda", generator=g).to(dt) for d in (dk, dv))
    la = -torch.rand(H, device="cuda", generator=g) * 0.2
    state = torch.randn(B, H, dk, dv, device="cuda", generator=g)
    was = state.clone()
    count = torch.full((B,), M, dtype=torch.int32, device="cuda")
    order = torch.arange(M - 1, -1, -1, dtype=torch.int32, device="cuda")
    path = order.repeat(B, 1) if with_path else None
    lla.linear_decode_commit(k, v, la, state, count, path)
    for b, h in ((0, 0), (B - 1, H - 1)):
        a = [x.double().cpu().numpy() for x in (k[b, h], v[b, h], la[h], was[b, h], state[b, h])]
        ref, size = R.linear_commit(*a[:4], order.tolist() if with_path else list(range(M)))
        # M + 1 sums; a weight's exponent is one product (2^-24 of up to 0.2 M), expf four units
        R.tree_check(a[4], ref, size, "f32", M + 1, 0.2 * M + 4, (b, h))
    assert lla.device_error() == 0


# Dynamic shared memory of M (dk + dv) floats from just below to just above 48 KiB, which a kernel's static memory counts to.
@pytest.mark.parametrize("B,H,dk,dv,M", [
    (1, 2, 128, 64, 62), (1, 2, 128, 64, 64), (2, 1, 64, 64, 93), (2, 1, 64, 64, 96), (1, 1, 128, 128, 47), (1, 1, 128, 128, 48),
    (32, 32, 128, 64, 64), (32, 32, 128, 128, 47), (1, 3, 128, 63, 63), (1, 3, 128, 63, 64), (1, 1, 128, 128, 49),
])
def test_commits_around_48_kib(B, H, dk, dv, M):
    """Each size in a process of its own: a kernel that has been allowed more once is allowed it for good."""
    code = ("from tests.test_commit_shared_memory_gpu import commit_of\n"
            f"for d in ('bf16', 'f32'):\n  for p in (False, True): commit_of({B}, {H}, {M}, {dk}, {dv}, d, p)\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
