"""Thin ctypes binding of ``libeec.so`` (the C ABI declared in include/eec.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI.  PyTorch provides device memory and the current
stream.  The functions keep the C names without the ``eec_`` prefix.

The library must have been built in-tree (``python -m
equivariant_edge_convolution_amd.build``); without it the first call raises,
so nothing can silently fall back to another implementation.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libeec.so")

# status codes of include/eec.h
STATUS = {
    0: "EEC_OK", 1: "EEC_ERR_NULL", 2: "EEC_ERR_SHAPE", 3: "EEC_ERR_BOX", 4: "EEC_ERR_OUT_OF_BOX",
    5: "EEC_ERR_SPECIES", 6: "EEC_ERR_CAPACITY", 7: "EEC_ERR_ALIAS", 8: "EEC_ERR_WORKSPACE",
    9: "EEC_ERR_GEOMETRY", 10: "EEC_ERR_HIP",
}
EEC_ERR_CAPACITY = 6

# every entry point include/eec.h declares
SYMBOLS = (
    "eec_build_neighbors", "eec_neighbors_workspace_bytes", "eec_skin_check", "eec_radial_basis",
    "eec_radial_project", "eec_project_workspace_bytes", "eec_edge_message",
    "eec_energy_forces", "eec_energy_forces_folded", "eec_energy_forces_folded_noalloc",
    "eec_energy_forces_timed", "eec_workspace_bytes",
    "eec_radial_table_floats", "eec_radial_table_levels", "eec_radial_table_build", "eec_energy_forces_tabulated", "eec_last_error",
    "eec_add_rms_norm", "eec_add_rms_norm_backward", "eec_add_rms_norm_backward_workspace_bytes",
    "eec_linear", "eec_linear_workspace_bytes", "eec_linear_backward", "eec_linear_backward_workspace_bytes",
)
PHASES = ("prepare", "forward", "readout", "backward", "scatter")
VARIANTS = {"direct": 0, "folded": 1, "tabulated": 2}
DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.float8_e4m3fn: 3}
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}


class EECError(RuntimeError):
    def __init__(self, status: int, what: str, msg: str):
        super().__init__(f"{what}: {STATUS.get(status, status)}: {msg}")
        self.status = status
        self.name = STATUS.get(status, str(status))


class _Model(ctypes.Structure):
    _fields_ = [
        ("n_species", ctypes.c_int32), ("channels", ctypes.c_int32), ("n_basis", ctypes.c_int32),
        ("hidden", ctypes.c_int32), ("lmax", ctypes.c_int32), ("cutoff", ctypes.c_double),
        ("W1", ctypes.c_void_p), ("W2", ctypes.c_void_p), ("W3", ctypes.c_void_p),
        ("emb", ctypes.c_void_p), ("w_read", ctypes.c_void_p),
    ]


class _Graph(ctypes.Structure):
    _fields_ = [
        ("n_atoms", ctypes.c_int32), ("n_edges", ctypes.c_int64), ("row_ptr", ctypes.c_void_p),
        ("col", ctypes.c_void_p), ("shift", ctypes.c_void_p), ("rev", ctypes.c_void_p),
    ]


class _Table(ctypes.Structure):
    _fields_ = [("log2_pieces", ctypes.c_int32), ("coef", ctypes.c_void_p), ("level", ctypes.c_void_p)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libeec.so once and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m equivariant_edge_convolution_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, dbl, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double, ctypes.c_size_t
    P = ctypes.POINTER
    L.eec_last_error.restype = ctypes.c_char_p
    L.eec_last_error.argtypes = []
    L.eec_neighbors_workspace_bytes.restype = sz
    L.eec_neighbors_workspace_bytes.argtypes = [i32, P(dbl), dbl]
    L.eec_build_neighbors.restype = ctypes.c_int
    L.eec_build_neighbors.argtypes = [vp, i32, vp, P(dbl), dbl, vp, i32, i64, vp, vp, vp, vp, P(i64), vp, sz]
    L.eec_skin_check.restype = ctypes.c_int
    L.eec_skin_check.argtypes = [vp, i32, vp, vp, dbl, vp, vp]
    L.eec_radial_basis.restype = ctypes.c_int
    L.eec_radial_basis.argtypes = [vp, P(_Graph), vp, P(dbl), dbl, vp, vp, vp]
    L.eec_project_workspace_bytes.restype = sz
    L.eec_project_workspace_bytes.argtypes = [i32, i64, P(_Model)]
    L.eec_radial_project.restype = ctypes.c_int
    L.eec_radial_project.argtypes = [vp, P(_Graph), vp, P(_Model), vp, vp, vp, sz]
    L.eec_workspace_bytes.restype = sz
    L.eec_workspace_bytes.argtypes = [i32, i64, P(_Model)]
    L.eec_edge_message.restype = ctypes.c_int
    L.eec_edge_message.argtypes = [vp, P(_Graph), vp, P(dbl), vp, P(_Model), vp, vp, sz]
    L.eec_energy_forces.restype = ctypes.c_int
    L.eec_energy_forces.argtypes = [vp, P(_Graph), vp, P(dbl), vp, P(_Model), vp, vp, vp, vp, vp, sz]
    L.eec_energy_forces_folded.restype = ctypes.c_int
    L.eec_energy_forces_folded.argtypes = [vp, P(_Graph), vp, P(dbl), vp, P(_Model), vp, vp, vp, vp, vp, sz]
    L.eec_energy_forces_folded_noalloc.restype = ctypes.c_int
    L.eec_energy_forces_folded_noalloc.argtypes = [vp, P(_Graph), vp, P(dbl), vp, P(_Model), vp, vp, vp, vp]
    L.eec_energy_forces_timed.restype = ctypes.c_int
    L.eec_energy_forces_timed.argtypes = [vp, P(_Graph), vp, P(dbl), vp, P(_Model), vp, vp, vp, vp, vp, sz,
                                          i32, P(_Table), P(vp)]
    L.eec_energy_forces_tabulated.restype = ctypes.c_int
    L.eec_energy_forces_tabulated.argtypes = [vp, P(_Graph), vp, P(dbl), vp, P(_Model), P(_Table), vp, vp, vp,
                                              vp, vp, sz]
    L.eec_radial_table_floats.restype = sz
    L.eec_radial_table_floats.argtypes = [P(_Model), i32]
    L.eec_radial_table_build.restype = ctypes.c_int
    L.eec_radial_table_levels.restype = sz
    L.eec_radial_table_levels.argtypes = [P(_Model), i32]
    L.eec_radial_table_build.argtypes = [vp, P(_Model), i32, vp, sz, vp, vp]
    L.eec_add_rms_norm.restype = ctypes.c_int
    L.eec_add_rms_norm.argtypes = [vp, i64, i64, i32, vp, i64, vp, i64, vp, dbl, vp, vp, vp, vp]
    L.eec_add_rms_norm_backward_workspace_bytes.restype = sz
    L.eec_add_rms_norm_backward_workspace_bytes.argtypes = [i64, i64]
    L.eec_add_rms_norm_backward.restype = ctypes.c_int
    L.eec_add_rms_norm_backward.argtypes = [vp, i64, i64, i32, vp, i64, vp, i64, vp, vp, vp, i64, vp, vp, vp, sz]
    L.eec_linear_workspace_bytes.restype = sz
    L.eec_linear_workspace_bytes.argtypes = [i64, i64, i64, i32, i32]
    L.eec_linear.restype = ctypes.c_int
    L.eec_linear.argtypes = [vp, i64, i64, i64, i32, i32, vp, i64, vp, vp, i64, vp, vp, vp, i64, i32, vp, vp, vp, sz]
    L.eec_linear_backward_workspace_bytes.restype = sz
    L.eec_linear_backward_workspace_bytes.argtypes = [i64, i64, i64, i32, i32]
    L.eec_linear_backward.restype = ctypes.c_int
    L.eec_linear_backward.argtypes = [vp, i64, i64, i64, i32, i32, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, vp, sz]
    _lib = L
    return L


def _check(status: int, what: str):
    if status != 0:
        raise EECError(status, what, lib().eec_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _box(box) -> ctypes.Array:
    b = np.asarray(box, dtype=np.float64).reshape(3)
    return (ctypes.c_double * 3)(*b.tolist())


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _raw_stream(device: torch.device) -> int:
    """The current stream's handle (of a tensor's device), without torch's stream
    object: building that takes 1.9 us, the handle 0.1 us."""
    return torch._C._cuda_getCurrentRawStream(device.index)


@dataclass
class Model:
    """Model weights resident on the device (float32, contiguous)."""

    n_species: int
    channels: int
    cutoff: float
    W1: torch.Tensor
    W2: torch.Tensor
    W3: torch.Tensor
    emb: torch.Tensor
    w_read: torch.Tensor

    @classmethod
    def from_arrays(cls, m, device="cuda") -> "Model":
        f = lambda a: torch.as_tensor(np.ascontiguousarray(a, dtype=np.float32)).to(device)
        return cls(int(m.n_species), int(m.channels), float(m.cutoff), f(m.W1), f(m.W2), f(m.W3),
                   f(m.emb), f(m.w_read))

    def struct(self) -> _Model:
        return _Model(self.n_species, self.channels, 32, 64, 3, self.cutoff,
                      self.W1.data_ptr(), self.W2.data_ptr(), self.W3.data_ptr(),
                      self.emb.data_ptr(), self.w_read.data_ptr())


@dataclass
class Graph:
    """Receiver-sorted CSR on the device."""

    n_atoms: int
    n_edges: int
    row_ptr: torch.Tensor
    col: torch.Tensor
    shift: torch.Tensor
    rev: torch.Tensor

    @classmethod
    def from_arrays(cls, row_ptr, col, shift, rev, device="cuda") -> "Graph":
        t = lambda a, dt: torch.as_tensor(np.ascontiguousarray(a, dtype=dt)).to(device)
        return cls(len(row_ptr) - 1, len(col), t(row_ptr, np.int32), t(col, np.int32),
                   t(shift, np.int8).reshape(-1, 3), t(rev, np.int32))

    def struct(self) -> _Graph:
        return _Graph(self.n_atoms, self.n_edges, self.row_ptr.data_ptr(),
                      self.col.data_ptr() if self.n_edges else None,
                      self.shift.data_ptr() if self.n_edges else None,
                      self.rev.data_ptr() if self.n_edges else None)


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def _given(workspace: torch.Tensor, device) -> tuple[int, int]:
    """(address, bytes) of a caller's workspace, of any type, in this device's memory (a kernel would take a host
    address for its own)."""
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {device}, not on {workspace.device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def neighbors_workspace_bytes(n_atoms: int, box, cutoff: float) -> int:
    return int(lib().eec_neighbors_workspace_bytes(int(n_atoms), _box(box), float(cutoff)))


def workspace_bytes(n_atoms: int, n_edges: int, model: Model) -> int:
    m = model.struct()
    return int(lib().eec_workspace_bytes(int(n_atoms), int(n_edges), ctypes.byref(m)))


def project_workspace_bytes(n_atoms: int, n_edges: int, model: Model) -> int:
    m = model.struct()
    return int(lib().eec_project_workspace_bytes(int(n_atoms), int(n_edges), ctypes.byref(m)))


def build_neighbors(pos: torch.Tensor, box, cutoff: float, species: torch.Tensor | None = None,
                    n_species: int = 0, edge_capacity: int | None = None) -> Graph:
    """eec_build_neighbors; retries once with the exact capacity it reports."""
    dev = pos.device
    n = int(pos.shape[0])
    ws = _workspace(neighbors_workspace_bytes(n, box, cutoff), dev)
    cap = int(edge_capacity) if edge_capacity is not None else 200 * max(n, 1)
    for _ in range(2):
        row_ptr = torch.empty(n + 1, dtype=torch.int32, device=dev)
        col = torch.empty(max(cap, 1), dtype=torch.int32, device=dev)
        shift = torch.empty((max(cap, 1), 3), dtype=torch.int8, device=dev)
        rev = torch.empty(max(cap, 1), dtype=torch.int32, device=dev)
        ne = ctypes.c_int64(0)
        st = lib().eec_build_neighbors(_stream(dev), n, _ptr(pos), _box(box), float(cutoff),
                                       _ptr(species), int(n_species), cap, _ptr(row_ptr), _ptr(col),
                                       _ptr(shift), _ptr(rev), ctypes.byref(ne), _ptr(ws), ws.numel())
        if st == EEC_ERR_CAPACITY and edge_capacity is None:
            cap = int(ne.value)
            continue
        _check(st, "build_neighbors")
        E = int(ne.value)
        return Graph(n, E, row_ptr, col[:E], shift[:E], rev[:E])
    raise EECError(EEC_ERR_CAPACITY, "build_neighbors", "capacity retry failed")


class NeighborList:
    """Preallocated CSR buffers (``edge_capacity`` edges) and workspace for
    repeated eec_build_neighbors calls on one cell, e.g. the rebuilds of an MD
    loop, which may run on a side stream (the current stream at ``build``)."""

    def __init__(self, n_atoms: int, box, cutoff: float, edge_capacity: int, device,
                 species: torch.Tensor | None = None, n_species: int = 0):
        self.n, self.box, self.cutoff = int(n_atoms), box, float(cutoff)
        self.cap = int(edge_capacity)
        self.species, self.n_species = species, int(n_species)
        self.row_ptr = torch.empty(self.n + 1, dtype=torch.int32, device=device)
        self.col = torch.empty(max(self.cap, 1), dtype=torch.int32, device=device)
        self.shift = torch.empty((max(self.cap, 1), 3), dtype=torch.int8, device=device)
        self.rev = torch.empty(max(self.cap, 1), dtype=torch.int32, device=device)
        self.workspace = _workspace(neighbors_workspace_bytes(self.n, box, cutoff), device)

    def build(self, pos: torch.Tensor) -> Graph:
        """Build into the buffers on the current stream; returns a Graph view
        of them (its arrays are complete once that stream reaches this point)."""
        ne = ctypes.c_int64(0)
        st = lib().eec_build_neighbors(_stream(pos.device), self.n, _ptr(pos), _box(self.box), self.cutoff,
                                       _ptr(self.species), self.n_species, self.cap, _ptr(self.row_ptr),
                                       _ptr(self.col), _ptr(self.shift), _ptr(self.rev), ctypes.byref(ne),
                                       _ptr(self.workspace), self.workspace.numel())
        _check(st, "build_neighbors")
        E = int(ne.value)
        return Graph(self.n, E, self.row_ptr, self.col[:E], self.shift[:E], self.rev[:E])


def skin_check(pos: torch.Tensor, ref: torch.Tensor, half_skin: float, out=None):
    """eec_skin_check on the current stream: (max_r2 [1] float64, rebuild [1]
    int32), device tensors, nothing synchronised."""
    dev = pos.device
    m2, flag = out if out is not None else (torch.empty(1, dtype=torch.float64, device=dev),
                                            torch.empty(1, dtype=torch.int32, device=dev))
    _check(lib().eec_skin_check(_stream(dev), int(pos.shape[0]), _ptr(pos), _ptr(ref), float(half_skin),
                                _ptr(m2), _ptr(flag)), "skin_check")
    return m2, flag


def radial_basis(graph: Graph, pos: torch.Tensor, box, cutoff: float):
    dev = pos.device
    E = graph.n_edges
    r = torch.empty(E, dtype=torch.float32, device=dev)
    basis = torch.empty((E, 32), dtype=torch.float32, device=dev)
    Y = torch.empty((E, 16), dtype=torch.float32, device=dev)
    g = graph.struct()
    _check(lib().eec_radial_basis(_stream(dev), ctypes.byref(g), _ptr(pos), _box(box), float(cutoff),
                                  _ptr(r), _ptr(basis), _ptr(Y)), "radial_basis")
    return r, basis, Y


def radial_project(graph: Graph, species: torch.Tensor, model: Model, basis: torch.Tensor):
    dev = basis.device
    E = graph.n_edges
    R = torch.empty((E, 4 * model.channels), dtype=torch.float32, device=dev)
    ws = _workspace(project_workspace_bytes(graph.n_atoms, E, model), dev)
    g, m = graph.struct(), model.struct()
    _check(lib().eec_radial_project(_stream(dev), ctypes.byref(g), _ptr(species), ctypes.byref(m),
                                    _ptr(basis), _ptr(R), _ptr(ws), ws.numel()), "radial_project")
    return R


def edge_message(graph: Graph, pos: torch.Tensor, box, species: torch.Tensor, model: Model,
                 workspace: torch.Tensor | None = None, out: torch.Tensor | None = None):
    dev = pos.device
    n = graph.n_atoms
    A = out if out is not None else torch.empty((n, 16, model.channels), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = _workspace(workspace_bytes(n, graph.n_edges, model), dev)
    ws, size = _given(workspace, dev)
    g, m = graph.struct(), model.struct()
    _check(lib().eec_edge_message(_stream(dev), ctypes.byref(g), _ptr(pos), _box(box), _ptr(species),
                                  ctypes.byref(m), _ptr(A), ws, size), "edge_message")
    return A


class RadialTable:
    """eec_radial_table_build: the model's radial tables (device float32) and
    their certificate (device float64 [2]: value and r-derivative error
    relative to the local scale)."""

    def __init__(self, model: "Model", log2_pieces: int = 6):
        m = model.struct()
        n = int(lib().eec_radial_table_floats(ctypes.byref(m), int(log2_pieces)))
        nl = int(lib().eec_radial_table_levels(ctypes.byref(m), int(log2_pieces)))
        if n == 0 or nl == 0:
            raise EECError(2, "radial_table_build", "log2_pieces out of range")
        dev = model.W1.device
        self.log2_pieces = int(log2_pieces)
        self.coef = torch.empty(n, dtype=torch.float32, device=dev)
        self.level = torch.empty(nl, dtype=torch.int32, device=dev)
        self.certificate = torch.empty(2, dtype=torch.float64, device=dev)
        _check(lib().eec_radial_table_build(_stream(dev), ctypes.byref(m), self.log2_pieces, _ptr(self.coef), n,
                                            _ptr(self.level), _ptr(self.certificate)), "radial_table_build")

    def struct(self) -> _Table:
        return _Table(self.log2_pieces, self.coef.data_ptr(), self.level.data_ptr())


class EnergyForces:
    """Preallocated outputs + workspace for repeated eec_energy_forces calls."""

    def __init__(self, graph: Graph, model: Model, device, atom_energy=True, virial=False,
                 variant: str = "direct", edge_capacity: int | None = None, table: RadialTable | None = None):
        n = graph.n_atoms
        if (variant == "tabulated") != (table is not None):
            raise ValueError("the tabulated variant takes a RadialTable, the others none")
        self.table = table
        self._t = table.struct() if table is not None else None
        self.variant = VARIANTS[variant]
        self.graph, self.model = graph, model
        self.energy = torch.empty(1, dtype=torch.float32, device=device)
        self.atom_energy = torch.empty(n, dtype=torch.float32, device=device) if atom_energy else None
        self.forces = torch.empty((n, 3), dtype=torch.float32, device=device)
        self.virial = torch.empty((3, 3), dtype=torch.float32, device=device) if virial else None
        self.cap = max(graph.n_edges, 0 if edge_capacity is None else int(edge_capacity))
        self.workspace = _workspace(workspace_bytes(n, self.cap, model), device)
        self._g = graph.struct()
        self._m = model.struct()

    def __call__(self, pos: torch.Tensor, box, species: torch.Tensor, events=None, graph: Graph | None = None):
        """One eec_energy_forces call on the current stream; with ``events`` (a
        sequence of 2 * len(PHASES) hipEvent_t handles) the instrumented entry
        point records them around each phase.  ``graph`` replaces the bound
        list (same atoms, at most ``edge_capacity`` edges), e.g. after a rebuild."""
        if graph is not None:
            if graph.n_atoms != self.graph.n_atoms or graph.n_edges > self.cap:
                raise ValueError("graph does not fit this EnergyForces (atoms or edge capacity)")
            self.graph, self._g = graph, graph.struct()
        s = _stream(pos.device)
        args = (s, ctypes.byref(self._g), _ptr(pos), _box(box), _ptr(species), ctypes.byref(self._m),
                _ptr(self.energy), _ptr(self.atom_energy), _ptr(self.forces), _ptr(self.virial),
                _ptr(self.workspace), self.workspace.numel())
        tab = ctypes.byref(self._t) if self._t is not None else None
        if events is None:
            if self.variant == 2:
                _check(lib().eec_energy_forces_tabulated(*args[:6], tab, *args[6:]), "energy_forces_tabulated")
            else:
                fn = lib().eec_energy_forces if self.variant == 0 else lib().eec_energy_forces_folded
                _check(fn(*args), "energy_forces")
        else:
            arr = (ctypes.c_void_p * len(events))(*events)
            _check(lib().eec_energy_forces_timed(*args, self.variant, tab, arr), "energy_forces_timed")
        return self


def energy_forces(graph: Graph, pos: torch.Tensor, box, species: torch.Tensor, model: Model,
                  virial: bool = False, variant: str = "direct", table: RadialTable | None = None):
    """eec_energy_forces (variant "direct"), eec_energy_forces_folded ("folded")
    or eec_energy_forces_tabulated ("tabulated", with ``table``)."""
    ef = EnergyForces(graph, model, pos.device, atom_energy=True, virial=virial, variant=variant, table=table)
    ef(pos, box, species)
    out = dict(energy=ef.energy, atom_energy=ef.atom_energy, forces=ef.forces)
    if virial:
        out["virial"] = ef.virial
    return out


def energy_forces_folded_noalloc(graph: Graph, pos: torch.Tensor, box, species: torch.Tensor, model: Model,
                                 virial: bool = False, out: dict | None = None):
    """eec_energy_forces_folded_noalloc: the folded call with the library's
    static device scratch instead of a workspace.  `out` (energy, atom_energy,
    forces and optionally virial tensors, e.g. from an earlier call) is
    written in place; otherwise the outputs are allocated here (by torch, on
    the caller's side of the boundary)."""
    dev = pos.device
    n = graph.n_atoms
    if out is None:
        out = dict(energy=torch.empty(1, dtype=torch.float32, device=dev),
                   atom_energy=torch.empty(n, dtype=torch.float32, device=dev),
                   forces=torch.empty((n, 3), dtype=torch.float32, device=dev))
        if virial:
            out["virial"] = torch.empty((3, 3), dtype=torch.float32, device=dev)
    g, m = graph.struct(), model.struct()
    _check(lib().eec_energy_forces_folded_noalloc(_stream(dev), ctypes.byref(g), _ptr(pos), _box(box),
                                                  _ptr(species), ctypes.byref(m), _ptr(out["energy"]),
                                                  _ptr(out.get("atom_energy")), _ptr(out["forces"]),
                                                  _ptr(out.get("virial"))), "energy_forces_folded_noalloc")
    return out


def _matrix(t: torch.Tensor, name: str, rows: int, width: int, dtype, device) -> int:
    """Checks a [rows][width] matrix of adjacent columns; returns its row stride."""
    if t.shape != (rows, width):
        raise ValueError(f"{name} must be [{rows}][{width}], not {list(t.shape)}")
    if t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be {dtype} on {device}, not {t.dtype} on {t.device}")
    ld, step = t.stride()
    if step != 1 and width > 1:
        raise ValueError(f"the columns of {name} must be adjacent")
    return ld if rows > 1 else width


def _vector(t: torch.Tensor | None, name: str, n: int, dtype, device):
    """Checks a contiguous vector of n elements (or None); returns its address."""
    if t is None:
        return None
    if t.shape != (n,) or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be {n} contiguous elements of {dtype} on {device}")
    return t.data_ptr()


def _dense_input(t: torch.Tensor, name: str):
    """(rows, width, dtype, device) of an operator's first matrix."""
    if t.dim() != 2 or t.dtype not in DTYPES or not t.is_cuda:
        raise ValueError(f"{name} must be a device matrix of float32, float16, bfloat16 or (linear) float8_e4m3fn")
    return *t.shape, t.dtype, t.device


def _address(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=4096)
def _linear_workspace(rows: int, outer: int, inner: int, dtype: int, out_dtype: int) -> int:
    return lib().eec_linear_workspace_bytes(rows, outer, inner, dtype, out_dtype)


def _new_rows(like: torch.Tensor, rows: int, n: int) -> torch.Tensor:
    """A contiguous [rows][n] of the same type (empty_like, where it serves, is the quickest way to one)."""
    return torch.empty_like(like) if like.is_contiguous() else like.new_empty((rows, n))


def add_rms_norm(x: torch.Tensor, weight: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                 eps: float = 1e-6, quantize: bool = False, save_rstd: bool = False) -> dict:
    """eec_add_rms_norm on rows of ``x`` (any row stride): ``y``, ``sum`` (x +
    residual; x itself without a residual), with ``quantize`` ``y`` in
    float8_e4m3fn and its row ``scale``, with ``save_rstd`` ``rstd``."""
    rows, n, dt, dev = _dense_input(x, "x")
    ldx = _matrix(x, "x", rows, n, dt, dev)
    ldr = _matrix(residual, "residual", rows, n, dt, dev) if residual is not None else 0
    w = _vector(weight, "weight", n, dt, dev)
    y = torch.empty((rows, n), dtype=torch.float8_e4m3fn, device=dev) if quantize else _new_rows(x, rows, n)
    out = dict(y=y, sum=x)
    total = scale = rstd = None
    if residual is not None:
        total = out["sum"] = _new_rows(x, rows, n)
    if quantize:
        scale = out["scale"] = torch.empty(rows, dtype=torch.float32, device=dev)
    if save_rstd:
        rstd = out["rstd"] = torch.empty(rows, dtype=torch.float32, device=dev)
    _check(lib().eec_add_rms_norm(_raw_stream(dev), rows, n, DTYPES[dt], x.data_ptr(), ldx, _address(residual), ldr, w,
                                  float(eps), _address(total), y.data_ptr(), _address(scale), _address(rstd)),
           "add_rms_norm")
    return out


def add_rms_norm_backward(gy: torch.Tensor, sum: torch.Tensor, weight: torch.Tensor | None, rstd: torch.Tensor,
                          gsum: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> dict:
    """eec_add_rms_norm_backward: ``gx`` (the gradient of x and of residual) and
    ``gweight`` (None without a weight), from the forward's ``sum`` and ``rstd``."""
    rows, n, dt, dev = _dense_input(sum, "sum")
    lds = _matrix(sum, "sum", rows, n, dt, dev)
    ldgy = _matrix(gy, "gy", rows, n, dt, dev)
    ldgs = _matrix(gsum, "gsum", rows, n, dt, dev) if gsum is not None else 0
    w = _vector(weight, "weight", n, dt, dev)
    rs = _vector(rstd, "rstd", rows, torch.float32, dev)
    gx = _new_rows(sum, rows, n)
    gw, ws, size = None, None, 0
    if workspace is not None:
        ws, size = _given(workspace, dev)
    if weight is not None:
        gw = torch.empty(n, dtype=dt, device=dev)
        if workspace is None:
            workspace = _workspace(lib().eec_add_rms_norm_backward_workspace_bytes(rows, n), dev)
            ws, size = workspace.data_ptr(), workspace.numel()
    _check(lib().eec_add_rms_norm_backward(_raw_stream(dev), rows, n, DTYPES[dt], gy.data_ptr(), ldgy, sum.data_ptr(),
                                           lds, w, rs, _address(gsum), ldgs, gx.data_ptr(), _address(gw), ws, size),
           "add_rms_norm_backward")
    return dict(gx=gx, gweight=gw)


def linear(x: torch.Tensor, w: torch.Tensor, bias: torch.Tensor | None = None, act: str = "none",
           residual: torch.Tensor | None = None, x_scale: torch.Tensor | None = None,
           w_scale: torch.Tensor | None = None, out_dtype: torch.dtype | None = None, save_preact: bool = False,
           workspace: torch.Tensor | None = None) -> dict:
    """eec_linear: ``y`` = act(x w^T + bias) + residual and, with
    ``save_preact``, ``preact`` (what act is applied to).  float8_e4m3fn
    operands take their row scales and ``out_dtype`` (bfloat16 by default)."""
    rows, k, dt, dev = _dense_input(x, "x")
    n = w.shape[0]
    ot = out_dtype if out_dtype is not None else (torch.bfloat16 if dt == torch.float8_e4m3fn else dt)
    if ot not in DTYPES or act not in ACTS:
        raise ValueError(f"unknown out_dtype {ot} or activation {act!r}")
    ldx = _matrix(x, "x", rows, k, dt, dev)
    ldw = _matrix(w, "w", n, k, dt, dev)
    ldr = _matrix(residual, "residual", rows, n, ot, dev) if residual is not None else 0
    xs = _vector(x_scale, "x_scale", rows, torch.float32, dev)
    wsc = _vector(w_scale, "w_scale", n, torch.float32, dev)
    b = _vector(bias, "bias", n, ot, dev)
    y = x.new_empty((rows, n)) if ot == dt else torch.empty((rows, n), dtype=ot, device=dev)
    out = dict(y=y)
    if save_preact:
        out["preact"] = torch.empty((rows, n), dtype=ot, device=dev)
    dt, ot = DTYPES[dt], DTYPES[ot]
    ws, size = None, 0
    if workspace is not None:
        ws, size = _given(workspace, dev)
    elif need := _linear_workspace(rows, n, k, dt, ot):
        workspace = _workspace(need, dev)
        ws, size = workspace.data_ptr(), need
    _check(lib().eec_linear(_raw_stream(dev), rows, n, k, dt, ot, x.data_ptr(), ldx, xs, w.data_ptr(),
                            ldw, wsc, b, _address(residual), ldr, ACTS[act], y.data_ptr(), _address(out.get("preact")),
                            ws, size), "linear")
    return out


def linear_backward(gy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, preact: torch.Tensor | None = None,
                    act: str = "none", bias: bool = True, workspace: torch.Tensor | None = None) -> dict:
    """eec_linear_backward: ``gx``, ``gw`` and, with ``bias``, ``gbias`` (the
    gradient of the residual is ``gy``)."""
    rows, k, dt, dev = _dense_input(x, "x")
    n = w.shape[0]
    if act not in ACTS:
        raise ValueError(f"unknown activation {act!r}")
    ldx = _matrix(x, "x", rows, k, dt, dev)
    ldw = _matrix(w, "w", n, k, dt, dev)
    ldgy = _matrix(gy, "gy", rows, n, dt, dev)
    if act != "none":
        if preact is None:
            raise ValueError("an activation's backward needs preact")
        _matrix(preact, "preact", rows, n, dt, dev)
        if not preact.is_contiguous():
            raise ValueError("preact must be contiguous")
    gx, gw = _new_rows(x, rows, k), _new_rows(w, n, k)
    gb = torch.empty(n, dtype=dt, device=dev) if bias else None
    if workspace is None:
        workspace = _workspace(lib().eec_linear_backward_workspace_bytes(rows, n, k, DTYPES[dt], ACTS[act]), dev)
    ws, size = _given(workspace, dev)
    _check(lib().eec_linear_backward(_raw_stream(dev), rows, n, k, DTYPES[dt], ACTS[act], gy.data_ptr(), ldgy,
                                     x.data_ptr(), ldx, w.data_ptr(), ldw, _address(preact), gx.data_ptr(),
                                     gw.data_ptr(), _address(gb), ws, size), "linear_backward")
    return dict(gx=gx, gw=gw, gbias=gb)


class HipEvents:
    """hipEvent_t handles from the HIP runtime, for timing phases on the stream
    the library launches on (torch's own events only see torch's launches)."""

    def __init__(self, n: int):
        self._hip = ctypes.CDLL("libamdhip64.so")
        self._hip.hipEventCreate.argtypes = [ctypes.POINTER(ctypes.c_void_p)]
        self._hip.hipEventElapsedTime.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.c_void_p, ctypes.c_void_p]
        self._hip.hipEventDestroy.argtypes = [ctypes.c_void_p]
        self.handles = []
        for _ in range(n):
            h = ctypes.c_void_p()
            if self._hip.hipEventCreate(ctypes.byref(h)) != 0:
                raise RuntimeError("hipEventCreate failed")
            self.handles.append(h.value)

    def elapsed_ms(self, a: int, b: int) -> float:
        ms = ctypes.c_float()
        if self._hip.hipEventElapsedTime(ctypes.byref(ms), self.handles[a], self.handles[b]) != 0:
            raise RuntimeError("hipEventElapsedTime failed")
        return float(ms.value)

    def close(self):
        for h in self.handles:
            self._hip.hipEventDestroy(h)
        self.handles = []
