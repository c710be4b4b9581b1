"""The paged-cache operators where what a call allows ends, without a GPU."""

import os
import shutil

from test_paged_cpu import A, INVALID, OK, _attend


def test_a_bound_above_the_tokens(lib):
    """A fixed bound is clipped to the tokens that there are, before what else is asked of it."""
    so = lib.load_library()
    for most in (1, 64, 65, 2 ** 40):
        assert _attend(so, tokens=0, most=most, starts=A) == OK, most
        assert _attend(so, tokens=0, most=most, starts=A, masks=A) == OK, most
        assert _attend(so, tokens=0, most=most) == INVALID          # without starts it is tokens / batch
    for kw in (dict(tokens=6, most=0), dict(tokens=6, most=-1), dict(tokens=0, most=-1), dict(tokens=-1, most=3),
               dict(tokens=65, most=65, masks=A), dict(tokens=65, most=100, masks=A)):
        assert _attend(so, starts=A, **kw) == INVALID, kw
        assert so.rope_last_error()


def test_a_binding_of_other_sources_is_not_loaded(tmp_path, monkeypatch):
    """The compiled short way carries what it was made of in its name: one of another header or another source is
    neither found nor returned, not even where the new one cannot be compiled."""
    from rotary_position_embedding_gb300 import build

    sources = []
    for f in build.BINDING_SOURCES:
        sources.append(shutil.copy(f, tmp_path))
    monkeypatch.setattr(build, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(build, "BINDING_SOURCES", tuple(sources))
    paths = [build.binding_path(sources, str(tmp_path))]
    assert os.path.basename(paths[0]) == os.path.basename(build.BINDING_PATH)
    for f in sources:
        with open(f, "a") as s:
            s.write("// more\n")
        paths.append(build.binding_path(sources, str(tmp_path)))
    assert len(set(paths)) == 3
    for path in paths[:2]:
        open(path, "w").close()
    monkeypatch.setenv("PATH", str(tmp_path / "none"))          # no g++
    assert build.build_binding() is None and not os.path.exists(paths[2])
    open(paths[2], "w").close()
    assert build.build_binding() == paths[2]                    # made of these sources
