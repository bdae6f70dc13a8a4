"""Host-only checks of calls of the paged cache at their edges."""
from test_kv_more_cpu import CUDA_ERR, FAKE, INVALID, NO_DEVICE, OK, _append_norm, _fork, lib  # noqa: F401  (lib is a fixture)


def test_a_batch_that_has_ended(lib):
    """No places go on: an array of no parents is a null pointer, which is not "every place goes on with itself"."""
    assert _fork(lib, B=0, parents=None) == OK                     # 16 places before
    assert _fork(lib, B=0, parents=None, room=None, out=None, out_lens=None) == OK
    assert _fork(lib, B=0) == OK
    assert _fork(lib, B=0, parents=None, room_all=-1) == INVALID
    assert _fork(lib, B=1, parents=None) == INVALID


@NO_DEVICE
def test_batches_that_go_on_pass_the_checks(lib):
    assert _fork(lib, B=16, parents=None) == CUDA_ERR
    assert _fork(lib, B=1) == CUDA_ERR


def test_norms_of_no_tokens(lib):
    """A step without new tokens: its queries' array may be a null pointer, with norms as without."""
    for q_norm in (None, FAKE + (12 << 32)):
        assert _append_norm(lib, T=0, B=0, k=None, v=None, q=None, q_out=None, q_norm=q_norm) == OK
        assert _append_norm(lib, T=0, B=3, cu=FAKE, k=None, v=None, q=None, q_out=None, q_norm=q_norm) == OK
    assert _append_norm(lib, q=None, q_out=None) == INVALID        # keys alone have no queries to norm
